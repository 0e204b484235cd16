// FP8 cache pages as bf16 pages, ahead of an attention of several row groups.
//
// A group of 128 query rows that reads FP8 pages converts them itself, in shared memory,
// at ~2.3 us per page and CTA pair (its converter warps are the bound) against ~0.95 us
// for a bf16 page.  Where a sequence has more than one group (trees: one per node at 128
// heads), every group would convert the same pages again; converting each page once into
// a scratch pool costs 656 bytes read and 1152 written per row and lets the groups read
// bf16 pages from the L2.  24 trees of up to 11 nodes x 128 heads over 256 .. 4096 rows:
// 220 us converted by group, 136 us ahead, of which the conversion takes 14 (9 for its bytes
// at the copy rate: a sequence has as many CTAs whatever its length, so that those of the
// long ones take three turns).  The values are the same: E4M3(code) * scale in fp32, rounded
// to bf16.
//
// Page p of sequence b becomes block b * max_pages + p of the scratch pool, and the
// scratch block table says so.  A warp takes a row at a time: lane l converts codes
// [16 l, 16 l + 16) (512 contiguous bytes in, 1024 out), lanes 0..7 move the RoPE values.
#include "mla_fp8.cuh"
#include "mla_internal.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kExpandThreads = 256;
constexpr int kRowsAtOnce = 4;    // rows a warp has in flight: a CTA's half page in one step
static_assert(kRowsAtOnce * (kExpandThreads / 32) == kPage / 2, "half a page per step");

struct ExpandArgs {
  const unsigned char* rows;
  int num_blocks;
  const int32_t* block_table;
  int bt_stride, max_pages;
  const int32_t* seq_lens;
  int checked;
  int* hdr;
  int32_t* table;
  unsigned char* pool;      // bf16 [B * max_pages, 64, 576]
};

__global__ void __launch_bounds__(kExpandThreads) fp8_expand_kernel(ExpandArgs a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t* row_blocks = a.block_table + (size_t)b * a.bt_stride;
  int blk = row_blocks[blockIdx.x >> 1];   // (asked for together with the length; blockIdx.x < 2 max_pages)
  int S = a.seq_lens[b];
  S = S < 0 ? 0 : min(S, a.max_pages * kPage);
  const int pages = (S + kPage - 1) / kPage;
  for (int half = blockIdx.x; half < 2 * pages; half += gridDim.x) {
    const int p = half >> 1, first = (half & 1) * (kPage / 2);
    if (half != (int)blockIdx.x) blk = row_blocks[p];
    const bool in_pool = blk >= 0 && blk < a.num_blocks;
    const size_t to = (size_t)b * a.max_pages + p;
    if (threadIdx.x == 0 && first == 0) {
      a.table[to] = (int)to;
      if (!in_pool && a.checked) record_error(a.hdr, MLA_ERR_DEVICE_CHECK, (b << 16) | p);
    }
    const int valid = min(first + kPage / 2, S - p * kPage);
    const unsigned char* src = a.rows + (in_pool ? (size_t)blk * kPage * kFp8RowBytes : 0);
    unsigned char* dst = a.pool + to * kPage * (2 * kDK);
    {
      const int r0 = first + warp;
      uint4 code[kRowsAtOnce], rope[kRowsAtOnce];
      float scale[kRowsAtOnce];
#pragma unroll
      for (int k = 0; k < kRowsAtOnce; ++k) {
        const int r = r0 + k * (kExpandThreads / 32);
        const unsigned char* row = src + (size_t)r * kFp8RowBytes;
        const bool read = r < valid && in_pool;      // (a block outside the pool reads as zeros)
        code[k] = read ? *reinterpret_cast<const uint4*>(row + 16 * lane) : make_uint4(0, 0, 0, 0);
        scale[k] = read ? *reinterpret_cast<const float*>(row + kDLat + 4 * (lane >> 3)) : 0.f;
        rope[k] = read && lane < 8 ? *reinterpret_cast<const uint4*>(row + kDLat + 16 + 16 * lane) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < kRowsAtOnce; ++k) {
        const int r = r0 + k * (kExpandThreads / 32);
        if (r >= valid) break;
        const uint64_t s2 = ((uint64_t)__float_as_uint(scale[k]) << 32) | __float_as_uint(scale[k]);
        const uint2 x = dequant4(code[k].x, s2), y = dequant4(code[k].y, s2);
        const uint2 z = dequant4(code[k].z, s2), w = dequant4(code[k].w, s2);
        unsigned char* out = dst + (size_t)r * (2 * kDK);
        const uint32_t v[8] = {x.x, x.y, y.x, y.y, z.x, z.y, w.x, w.y};
        ptx::st_global_v8(out + 32 * lane, v);
        if (lane < 8) *reinterpret_cast<uint4*>(out + 2 * kDLat + 16 * lane) = rope[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_fp8_expand(const Fp8Pool& pool, const int32_t* block_table, int bt_stride, int B, int max_pages,
                              const int32_t* seq_lens, int checked, void* ws, int32_t* table, void* out,
                              cudaStream_t st) {
  ExpandArgs a{pool.rows, pool.num_blocks, block_table, bt_stride, max_pages, seq_lens, checked,
               static_cast<int*>(ws), table, static_cast<unsigned char*>(out)};
  // about eight CTAs per SM, shared evenly by the sequences
  const int sms = mla_device_sm_count();
  long long gx = (8LL * (sms > 0 ? sms : 148) + B - 1) / B;
  if (gx > 2LL * max_pages) gx = 2LL * max_pages;
  return launch_pdl(fp8_expand_kernel, dim3((unsigned)gx, (unsigned)B), dim3(kExpandThreads), 0, st, a);
}

}  // namespace mla
