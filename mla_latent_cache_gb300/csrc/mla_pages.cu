// The pages of a paged cache: accepted rows moved together, sequences shortened,
// lengthened and forked, pages copied.
//
// Bookkeeping lives on the device next to the block table: refs[k] is the number of
// block-table entries that hold block k (0: free).  Whatever is allocated is the lowest
// free blocks in order (sequence by sequence, page by page; fork by fork), so that the
// result is a function of the arguments alone: counts change by integer atomics, whose
// order does not show, and free blocks are ranked by a block-wide scan.
//
// Bound: the row moves and page copies by memory (each moved byte is read and written
// once); the bookkeeping by latency (one CTA: a few thousand integers).
#include <algorithm>

#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kBookThreads = 1024;    // the bookkeeping kernels' one CTA
constexpr int kScanPerThread = 16;    // refs entries per thread and step of the free-block scan
constexpr int kCopyThreads = 256;
constexpr int kCompactThreads = 512;
constexpr int kMaxCompactSplit = 8;   // CTAs per sequence at most
constexpr int kItems = 8;             // 16-byte pieces a thread holds at once in a row move

// A pool as rows of 16-byte pieces in one or two parts: 64 latent + 8 RoPE pieces of a
// bf16 row, or 41 pieces of a 656-byte FP8 row.
struct RowPool {
  char *part0, *part1;
  int64_t row0, block0, row1, block1;   // strides, bytes
  int num_blocks;
};
template <int kCols0, int kCols1>
__device__ __forceinline__ char* piece(const RowPool& p, int row, int col) {
  const int64_t blk = row / kPage, j = row % kPage;
  if (kCols1 == 0 || col < kCols0) return p.part0 + blk * p.block0 + j * p.row0 + 16 * col;
  return p.part1 + blk * p.block1 + j * p.row1 + 16 * (col - kCols0);
}

__device__ __forceinline__ void report(int* status) { atomicCAS(status, 0, MLA_ERR_DEVICE_CHECK); }

// Block-wide exclusive scan of one int per thread; *total gets the block's sum.  sh: 33 ints.
__device__ int block_excl_scan(int v, int* total, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < nwarps ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sh[lane] = w;
  }
  __syncthreads();
  const int pre = warp ? sh[warp - 1] : 0;
  *total = sh[nwarps - 1];
  __syncthreads();
  return pre + x - v;
}

// This thread's refs entries of the scan step that starts at block `base`.
struct RefsChunk {
  int v[kScanPerThread];
};
__device__ __forceinline__ RefsChunk load_refs(const int32_t* refs, int num_blocks, int base) {
  const int k0 = base + threadIdx.x * kScanPerThread;
  RefsChunk c;
#pragma unroll
  for (int g = 0; g < kScanPerThread; g += 4) {
    if (k0 + g + 4 <= num_blocks) {
      const int4 u = __ldcg(reinterpret_cast<const int4*>(refs + k0 + g));
      c.v[g] = u.x; c.v[g + 1] = u.y; c.v[g + 2] = u.z; c.v[g + 3] = u.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) c.v[g + e] = k0 + g + e < num_blocks ? __ldcg(refs + k0 + g + e) : 1;
    }
  }
  return c;
}

// take(rank, block) for the `want` lowest free blocks, ranks 0 .. in block order; returns
// how many there were.  chunk: the entries from block 0 on, loaded by the caller.  refs
// entries taken here are written by `take` itself.
template <typename Take>
__device__ int take_free(const int32_t* refs, int num_blocks, int want, int* sh, RefsChunk chunk, Take take) {
  int found = 0;
  for (int base = 0; base < num_blocks && found < want; base += kBookThreads * kScanPerThread) {
    const int k0 = base + threadIdx.x * kScanPerThread;
    if (base > 0) chunk = load_refs(refs, num_blocks, base);
    const int (&v)[kScanPerThread] = chunk.v;
    int mine = 0;
#pragma unroll
    for (int g = 0; g < kScanPerThread; ++g) mine += v[g] == 0;
    int total;
    int rank = found + block_excl_scan(mine, &total, sh);
#pragma unroll
    for (int g = 0; g < kScanPerThread; ++g) {
      if (v[g] == 0) {
        if (rank < want) take(rank, k0 + g);
        ++rank;
      }
    }
    found += total;
  }
  return found < want ? found : want;
}

// ------------------------------------------------------------------ accepted rows moved together
struct CompactArgs {
  RowPool pool;
  const int32_t* block_table;
  int bt_stride, max_pages;
  const int32_t *seq_lens, *node_lens, *accept_len, *accept_idx;
  int T;
  int32_t* new_lens;
  int* status;
};

// Accepted node idx[i] moves to place i; idx rises strictly, so idx[i] >= i: rows are taken
// in runs, all of a run's pieces held in registers before any is written, and a later run's
// sources (idx[j] >= j) lie past an earlier run's places.  Columns of pieces do not meet, so
// that a sequence's are shared out to as many CTAs (gridDim.y) as there is room for.
// 512 threads, two CTAs per SM: 256 sequences of up to 48 accepted rows 5.9 us with 256
// threads, 4.3 with 512; 128 sequences of up to 1000 rows 112 us with one CTA of 256 threads
// each, 53 with one of 512, 37 with two; 32 sequences of up to 200 rows 9.8 us with one, 3.9
// with eight.
template <int kCols0, int kCols1, bool kSplit>
__global__ void __launch_bounds__(kCompactThreads, 2) compact_kernel(CompactArgs a) {
  constexpr int kCols = kCols0 + kCols1;
  extern __shared__ int rows[];          // source and destination row of each accepted node
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int32_t* idx = a.accept_idx + (size_t)b * a.T;
  // (a thread's first node is asked for together with the lengths)
  const int t_first = tid < a.T ? idx[tid] : 0, prev_first = tid > 0 && tid < a.T ? idx[tid - 1] : -1;
  const int S = a.seq_lens[b], n = a.node_lens ? a.node_lens[b] : a.T, acc = a.accept_len[b];
  bool bad = n < 0 || n > a.T || S < n || S > a.max_pages * kPage || acc < 0 || acc > n;
  if (!bad) {
    for (int i = tid; i < acc; i += kCompactThreads) {
      const int t = i == tid ? t_first : idx[i], prev = i == tid ? prev_first : idx[i - 1];
      if (t <= prev || t >= n) { bad = true; continue; }
      const int from = S - n + t, to = S - n + i;
      const int bf = a.block_table[(size_t)b * a.bt_stride + from / kPage];
      const int bt = a.block_table[(size_t)b * a.bt_stride + to / kPage];
      if (bf < 0 || bf >= a.pool.num_blocks || bt < 0 || bt >= a.pool.num_blocks) { bad = true; continue; }
      rows[2 * i] = bf * kPage + from % kPage;
      rows[2 * i + 1] = bt * kPage + to % kPage;
    }
  }
  if (__syncthreads_or(bad)) {            // nothing of this sequence is moved
    if (tid == 0) {
      report(a.status);
      if (blockIdx.y == 0) a.new_lens[b] = S;
    }
    return;
  }
  if (tid == 0 && blockIdx.y == 0) a.new_lens[b] = S - n + acc;
  const int col0 = kSplit ? kCols * blockIdx.y / gridDim.y : 0;
  const int width = kSplit ? kCols * (blockIdx.y + 1) / gridDim.y - col0 : kCols;
  const int items = acc * width;
  // i / width for i < 1024 * kCols < 2^17: width < 2^7 is off by less than 2^-15 in 1 / width
  const unsigned inv = 0xffffffffu / width + 1;
  for (int base = 0; base < items; base += kCompactThreads * kItems) {
    uint4 v[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int it = base + k * kCompactThreads + tid, i = kSplit ? (int)__umulhi(it, inv) : it / kCols;
      if (it < items) v[k] = *reinterpret_cast<const uint4*>(piece<kCols0, kCols1>(a.pool, rows[2 * i], col0 + it - i * width));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int it = base + k * kCompactThreads + tid, i = kSplit ? (int)__umulhi(it, inv) : it / kCols;
      if (it < items && rows[2 * i] != rows[2 * i + 1])
        *reinterpret_cast<uint4*>(piece<kCols0, kCols1>(a.pool, rows[2 * i + 1], col0 + it - i * width)) = v[k];
    }
  }
}

// ------------------------------------------------------------------ sequences shortened and lengthened
struct ResizeArgs {
  int32_t* refs;
  int num_blocks;
  int32_t* block_table;
  int bt_stride, max_pages;
  const int32_t *cur_lens, *new_lens;
  int B;
  int32_t* got_lens;
  int* status;
};

// The last index of the non-decreasing v[0 .. n) with v[index] <= x (v[0] <= x).
__device__ __forceinline__ int last_at_most(const int* v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ int pages_of(int len) { return (int)(((long long)len + kPage - 1) / kPage); }

__global__ void __launch_bounds__(kBookThreads) resize_kernel(ResizeArgs a) {
  extern __shared__ int first[];       // [B]: pages asked for by the sequences before b
  __shared__ int sh[33], back_first[kBookThreads], back_page[kBookThreads];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int max_rows = a.max_pages * kPage;
  // For 1024 sequences at a time: the pages to give back and those asked for, counted and
  // ranked in sequence order; then the former, one page per thread.
  int want = 0;
  for (int base = 0; base < a.B; base += kBookThreads) {
    const int b = base + tid;
    int need = 0, back = 0, keep = 0;
    if (b < a.B) {
      const int cur = a.cur_lens[b], len = a.new_lens[b];
      if (cur < 0 || cur > max_rows || len < 0 || len > max_rows) {
        report(a.status);
      } else {
        keep = pages_of(len);
        need = max(0, keep - pages_of(cur));
        back = max(0, pages_of(cur) - keep);
      }
    }
    int total_need, total_back;
    const int pre_need = block_excl_scan(need, &total_need, sh);
    const int pre_back = block_excl_scan(back, &total_back, sh);
    if (b < a.B) first[b] = want + pre_need;
    want += total_need;
    back_first[tid] = pre_back;
    back_page[tid] = keep;
    __syncthreads();
    for (int i = tid; i < total_back; i += kBookThreads) {
      const int j = last_at_most(back_first, kBookThreads, i);
      int32_t* entry = a.block_table + (size_t)(base + j) * a.bt_stride + back_page[j] + (i - back_first[j]);
      const int k = *entry;
      *entry = -1;
      if (k < 0 || k >= a.num_blocks) {
        report(a.status);
      } else if (atomicSub(&a.refs[k], 1) <= 0) {   // held by nobody: the count stays at 0
        atomicAdd(&a.refs[k], 1);
        report(a.status);
      }
    }
    __syncthreads();
  }
  __threadfence();
  __syncthreads();
  const RefsChunk chunk = want == 0 ? RefsChunk{} : load_refs(a.refs, a.num_blocks, 0);
  const int got = want == 0 ? 0 : take_free(a.refs, a.num_blocks, want, sh, chunk, [&](int rank, int k) {
    const int lo = last_at_most(first, a.B, rank);
    a.block_table[(size_t)lo * a.bt_stride + pages_of(a.cur_lens[lo]) + rank - first[lo]] = k;
    a.refs[k] = 1;
  });
  if (got < want && tid == 0) report(a.status);
  __syncthreads();                     // cur_lens may be got_lens: every rank is placed
  for (int b = tid; b < a.B; b += kBookThreads) {
    const int cur = a.cur_lens[b], len = a.new_lens[b];
    int held = len;
    if (cur < 0 || cur > max_rows || len < 0 || len > max_rows) {
      held = cur;
    } else {
      const int c = pages_of(cur), need = max(0, pages_of(len) - c);
      const int granted = max(0, min(need, got - first[b]));
      if (granted < need) {
        held = (c + granted) * kPage;
        for (int p = c + granted; p < c + need; ++p) a.block_table[(size_t)b * a.bt_stride + p] = -1;
      }
    }
    a.got_lens[b] = held;
  }
}

// ------------------------------------------------------------------ forks
struct ForkArgs {
  int32_t* refs;
  int num_blocks;
  int32_t* block_table;
  int bt_stride, max_pages;
  int32_t* seq_lens;
  int B;
  const int32_t *src, *dst;
  int F;
  int32_t* copies;     // [3, F]: from block, to block, rows
  int apply;           // the deciding kernel applies the forks too
  int* status;
};

// What fork f does to page p of its destination's table row (p < max_pages), to the counts
// and to its length.  One thread per (f, p); a fork from itself has work at one page only.
__device__ __forceinline__ void fork_apply(const ForkArgs& a, int f, int p) {
  const int from = a.copies[f], to = a.copies[a.F + f], rows = a.copies[2 * a.F + f];
  if (from == -2) return;
  const int s = a.src[f], d = a.dst[f];
  const int len = a.seq_lens[s], full = len / kPage;
  int32_t* out = a.block_table + (size_t)d * a.bt_stride;
  if (s == d) {
    if (rows && p == full) {
      atomicSub(&a.refs[from], 1);
      out[p] = to;
    }
    return;
  }
  int k = -1;
  if (p < full) {
    k = a.block_table[(size_t)s * a.bt_stride + p];
    if (k >= 0 && k < a.num_blocks) atomicAdd(&a.refs[k], 1);
    else report(a.status);
  } else if (p == full && rows) {
    k = to;
  }
  out[p] = k;
  if (p == 0) a.seq_lens[d] = len;
}

// Up to this many (fork, page) pairs (eight per thread) are applied by the deciding CTA,
// more by a kernel of their own.  Release and fork of 48 sequences of 34 pages: 10.6 us in
// one kernel, 10.9 us and a launch more on the host in two.
constexpr int kApplyInPlan = 8192;

// Decides (one CTA): which forks stand, and the block of each copied last page.
// copies[f] = (from, to, rows) of the page to copy; rows 0: none; from -2: not forked.
__global__ void __launch_bounds__(kBookThreads) fork_plan_kernel(ForkArgs a) {
  extern __shared__ int dyn[];         // rank -> fork [F]; bits of rows that are a destination, and of those named twice
  __shared__ int sh[33];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int words = (a.B + 31) / 32;
  int* fork_of = dyn;
  unsigned* once = reinterpret_cast<unsigned*>(dyn + a.F);
  unsigned* twice = once + words;
  // (the scan's first blocks are on their way while the forks are looked at: no fork's
  // decision writes a count)
  const RefsChunk chunk = load_refs(a.refs, a.num_blocks, 0);
  for (int w = tid; w < 2 * words; w += kBookThreads) once[w] = 0;
  __syncthreads();
  for (int f = tid; f < a.F; f += kBookThreads) {
    const int d = a.dst[f];
    if (d < 0 || d >= a.B) continue;
    const unsigned bit = 1u << (d & 31);
    if (atomicOr(&once[d >> 5], bit) & bit) atomicOr(&twice[d >> 5], bit);
  }
  __syncthreads();
  int want = 0;
  for (int base = 0; base < a.F; base += kBookThreads) {
    const int f = base + tid;
    int need = 0;
    if (f < a.F) {
      const int s = a.src[f], d = a.dst[f];
      bool ok = s >= 0 && s < a.B && d >= 0 && d < a.B && !((twice[d >> 5] >> (d & 31)) & 1u);
      // a row that another fork overwrites is no source (itself: its last page is made its own)
      if (ok && s != d) ok = !((once[s >> 5] >> (s & 31)) & 1u);
      int from = -2, rows = 0;
      if (ok) {
        const int len = a.seq_lens[s];
        if (len < 0 || len > a.max_pages * kPage) {
          ok = false;
        } else {
          from = -1;
          const int tail = len % kPage;
          if (tail) {
            const int k = a.block_table[(size_t)s * a.bt_stride + len / kPage];
            if (k < 0 || k >= a.num_blocks) {
              ok = false;
              from = -2;
            } else if (s != d || a.refs[k] > 1) {
              from = k;
              rows = tail;
              need = 1;
            }
          }
        }
      }
      if (!ok) report(a.status);
      a.copies[f] = from;
      a.copies[a.F + f] = -1;
      a.copies[2 * a.F + f] = rows;
    }
    int total;
    const int rank = want + block_excl_scan(need, &total, sh);
    if (need) fork_of[rank] = f;
    want += total;
  }
  __syncthreads();
  const int got = want == 0 ? 0 : take_free(a.refs, a.num_blocks, want, sh, chunk, [&](int rank, int k) {
    a.copies[a.F + fork_of[rank]] = k;
    a.refs[k] = 1;
  });
  if (got < want) {                    // no block is left for the last forks
    if (tid == 0) report(a.status);
    for (int r = got + tid; r < want; r += kBookThreads) {
      a.copies[fork_of[r]] = -2;
      a.copies[2 * a.F + fork_of[r]] = 0;
    }
  }
  if (a.apply) {
    __syncthreads();
    for (int i = tid; i < a.F * a.max_pages; i += kBookThreads) fork_apply(a, i / a.max_pages, i % a.max_pages);
  }
}

// Applies (one CTA per fork).
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(ForkArgs a) {
  pdl_wait();
  pdl_trigger();
  for (int p = threadIdx.x; p < a.max_pages; p += kCopyThreads) fork_apply(a, blockIdx.x, p);
}

// ------------------------------------------------------------------ page copies
struct CopyArgs {
  RowPool pool;
  const int32_t* copies;    // [3, n]
  int n;
  int* status;
};

// Three CTAs per page share its first `rows` rows, each one step of kItems pieces per thread
// (48 half pages: 2.9 us, with one CTA each 4.0).
constexpr int kCopySplit = (kPage * 72 + kCopyThreads * kItems - 1) / (kCopyThreads * kItems);
template <int kCols0, int kCols1>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyArgs a) {
  constexpr int kCols = kCols0 + kCols1;
  pdl_wait();
  pdl_trigger();
  const int f = blockIdx.x, tid = threadIdx.x;
  const int from = a.copies[f], to = a.copies[a.n + f], rows = a.copies[2 * a.n + f];
  if (rows == 0) return;
  if (rows < 0 || rows > kPage || from < 0 || from >= a.pool.num_blocks || to < 0 || to >= a.pool.num_blocks) {
    if (tid == 0 && blockIdx.y == 0) report(a.status);
    return;
  }
  const int items = rows * kCols;
  const int base = blockIdx.y * kCopyThreads * kItems + tid;
  uint4 v[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int it = base + k * kCopyThreads;
    if (it < items) v[k] = *reinterpret_cast<const uint4*>(piece<kCols0, kCols1>(a.pool, from * kPage + it / kCols, it % kCols));
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int it = base + k * kCopyThreads;
    if (it < items) *reinterpret_cast<uint4*>(piece<kCols0, kCols1>(a.pool, to * kPage + it / kCols, it % kCols)) = v[k];
  }
}

RowPool row_pool(const CacheView& cv, unsigned char* rows_fp8) {
  RowPool p{};
  p.num_blocks = cv.num_blocks;
  if (rows_fp8) {
    p.part0 = reinterpret_cast<char*>(rows_fp8);
    p.row0 = 656;
    p.block0 = 656 * kPage;
  } else {
    p.part0 = reinterpret_cast<char*>(const_cast<__nv_bfloat16*>(cv.ckv));
    p.part1 = reinterpret_cast<char*>(const_cast<__nv_bfloat16*>(cv.kpe));
    p.row0 = cv.ckv_row * 2; p.block0 = cv.ckv_block * 2;
    p.row1 = cv.kpe_row * 2; p.block1 = cv.kpe_block * 2;
  }
  return p;
}

}  // namespace

cudaError_t launch_cache_compact(const CacheView& cv, unsigned char* rows_fp8, const int32_t* block_table,
                                 int bt_stride, int max_pages, const int32_t* seq_lens, const int32_t* node_lens,
                                 const int32_t* accept_len, const int32_t* accept_idx, int B, int T, int32_t* new_lens,
                                 cudaStream_t st) {
  CompactArgs a{row_pool(cv, rows_fp8), block_table, bt_stride, max_pages, seq_lens, node_lens, accept_len, accept_idx,
                T, new_lens, bmm_status_ptr()};
  if (!a.status) return cudaErrorInvalidValue;
  // as many CTAs per sequence as stay resident and can have a piece per thread
  long long split = 2LL * mla_device_sm_count() / B;
  const long long useful = (long long)T * (rows_fp8 ? 41 : 72) / kCompactThreads;
  split = std::max(1LL, std::min({split, useful, (long long)kMaxCompactSplit}));
  const size_t smem = (size_t)T * 2 * sizeof(int);
  const dim3 grid(B, (unsigned)split);
  const dim3 block(kCompactThreads);
  if (rows_fp8)
    return split > 1 ? launch_pdl(compact_kernel<41, 0, true>, grid, block, smem, st, a)
                     : launch_pdl(compact_kernel<41, 0, false>, grid, block, smem, st, a);
  return split > 1 ? launch_pdl(compact_kernel<64, 8, true>, grid, block, smem, st, a)
                   : launch_pdl(compact_kernel<64, 8, false>, grid, block, smem, st, a);
}

cudaError_t launch_pages_resize(int32_t* refs, int num_blocks, int32_t* block_table, int bt_stride, int max_pages,
                                const int32_t* cur_lens, const int32_t* new_lens, int B, int32_t* got_lens,
                                cudaStream_t st) {
  ResizeArgs a{refs, num_blocks, block_table, bt_stride, max_pages, cur_lens, new_lens, B, got_lens, bmm_status_ptr()};
  if (!a.status) return cudaErrorInvalidValue;
  return launch_pdl(resize_kernel, dim3(1), dim3(kBookThreads), (size_t)B * sizeof(int), st, a);
}

cudaError_t launch_pages_fork(int32_t* refs, int num_blocks, int32_t* block_table, int bt_stride, int max_pages,
                              int32_t* seq_lens, int B, const int32_t* src, const int32_t* dst, int F,
                              int32_t* copies, cudaStream_t st) {
  const bool apply = (long long)F * max_pages <= kApplyInPlan;
  ForkArgs a{refs, num_blocks, block_table, bt_stride, max_pages, seq_lens, B, src, dst, F, copies, apply,
             bmm_status_ptr()};
  if (!a.status) return cudaErrorInvalidValue;
  const size_t smem = ((size_t)F + 2 * (((size_t)B + 31) / 32)) * sizeof(int);
  const cudaError_t e = launch_pdl(fork_plan_kernel, dim3(1), dim3(kBookThreads), smem, st, a);
  return e != cudaSuccess || apply ? e : launch_pdl(fork_apply_kernel, dim3(F), dim3(kCopyThreads), 0, st, a);
}

cudaError_t launch_cache_copy(const CacheView& cv, unsigned char* rows_fp8, const int32_t* copies, int n,
                              cudaStream_t st) {
  CopyArgs a{row_pool(cv, rows_fp8), copies, n, bmm_status_ptr()};
  if (!a.status) return cudaErrorInvalidValue;
  const dim3 grid(n, kCopySplit);
  return rows_fp8 ? launch_pdl(copy_kernel<41, 0>, grid, dim3(kCopyThreads), 0, st, a)
                  : launch_pdl(copy_kernel<64, 8>, grid, dim3(kCopyThreads), 0, st, a);
}

}  // namespace mla
