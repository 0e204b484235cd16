// Device split planner: builds the work plan (segments, ranges, merge list) in
// the workspace from the device-resident sequence lengths, with no host sync.
// The rule is stated in include/mla.h next to the plan layout.
#include <climits>

#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kPlanThreads = 1024;

// Trees: the least pages of a range.  A range's first page is in its pair's hands after
// ~6 us whatever its length, and every further one takes ~0.9 us, against the merge of
// more parts (one tree of 8 nodes x 16 heads over 512 rows, decode: 4 pages 16.0 us, 2
// pages 14.4, 1 page 13.6; 4 nodes x 128 heads over 850 rows, plan and decode: 21.9, 20.9,
// 21.9).
constexpr int kTreeMinSplitPages = 2;
// Trees: the least threads of the planner.  A group, and as a rule a segment, per thread,
// and as few threads as that takes for cheap barriers (one group 4.0 us with 256 threads,
// 4.9 with 1024; 264 groups 5.9 with 512, 6.3 with 1024; 512 groups 9.9 with 256, 8.6 with
// 512, 8.4 with 1024: all with the groups' records read back from the workspace; where they
// stay in registers 3.8, 4.8 with 512 and 6.3 with 1024).
constexpr int kTreePlanThreads = 256;

constexpr int kSmemGroups = 4096;   // groups whose segment bases the planner keeps in shared memory

// Block-wide exclusive scans of three ints per thread at once; tot[] gets the
// block sums.  sh holds 3 x 32 ints.
__device__ void block_excl_scan3(int (&v)[3], int (&tot)[3], int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nwarps = blockDim.x >> 5;
  int x[3] = {v[0], v[1], v[2]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int y = __shfl_up_sync(0xffffffffu, x[j], o);
      if (lane >= o) x[j] += y;
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int j = 0; j < 3; ++j) sh[32 * j + warp] = x[j];
  }
  __syncthreads();
  if (warp < 3) {
    int w = lane < nwarps ? sh[32 * warp + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sh[32 * warp + lane] = w;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int pre = warp ? sh[32 * j + warp - 1] : 0;
    tot[j] = sh[32 * j + nwarps - 1];
    v[j] = pre + x[j] - v[j];
  }
  __syncthreads();
}

// Block-wide (sum, max) of two ints and (wrapping sum, min) of an unsigned and
// an int: warp shuffles, then one value per warp through shared memory.
__device__ void block_reduce(unsigned& usum, int& imin, int& isum, int& imax, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nwarps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    usum += __shfl_xor_sync(0xffffffffu, usum, o);
    imin = min(imin, __shfl_xor_sync(0xffffffffu, imin, o));
    isum += __shfl_xor_sync(0xffffffffu, isum, o);
    imax = max(imax, __shfl_xor_sync(0xffffffffu, imax, o));
  }
  if (lane == 0) {
    sh[warp] = (int)usum; sh[32 + warp] = imin; sh[64 + warp] = isum; sh[96 + warp] = imax;
  }
  __syncthreads();
  if (warp == 0) {
    usum = lane < nwarps ? (unsigned)sh[lane] : 0u;
    imin = lane < nwarps ? sh[32 + lane] : INT_MAX;
    isum = lane < nwarps ? sh[64 + lane] : 0;
    imax = lane < nwarps ? sh[96 + lane] : INT_MIN;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      usum += __shfl_xor_sync(0xffffffffu, usum, o);
      imin = min(imin, __shfl_xor_sync(0xffffffffu, imin, o));
      isum += __shfl_xor_sync(0xffffffffu, isum, o);
      imax = max(imax, __shfl_xor_sync(0xffffffffu, imax, o));
    }
    // (the shuffles follow every lane's reads, so lane 0 may overwrite the slots)
    if (lane == 0) {
      sh[0] = (int)usum; sh[1] = imin; sh[2] = isum; sh[3] = imax;
    }
  }
  __syncthreads();
  usum = (unsigned)sh[0]; imin = sh[1]; isum = sh[2]; imax = sh[3];
  __syncthreads();
}

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16; x *= 0x7feb352dU; x ^= x >> 15; x *= 0x846ca68bU; x ^= x >> 16;
  return x;
}

struct PlanArgs {
  const int32_t* seq_lens;   // length of sequence b is seq_lens[b / seq_div]
  int seq_div;               // 1; the sparse decode's S_q (one length per sequence, shared by its tokens)
  int B, T, H, causal, G, N, max_pages;
  int max_rows;              // longest allowed length: max_pages * 64, or the sparse decode's topk
  int RB, num_groups;
  int tree;                  // trees of drafted tokens: sequence b has node_lens[b] query tokens (null: T)
  const int32_t* node_lens;
  WsLayout L;
};

// Fixed cost of starting a group's work in a range, in pages (query staging and
// an output write per segment: measured ~8 us per segment change on the ragged
// V3 batch against ~0.8 us per page): the balanced ranges leave that many line
// positions between consecutive non-empty groups.
constexpr int kSegmentCostPages = 8;

// Segment s of a group with n pages whose first page sits at line position u
// (mode 1) and whose first segment is sb, in the given mode; writes the record
// and the range pointer of every range whose first segment it is (in mode 1
// also of the ranges inside the gap before it, which hold no segment).  ne:
// non-empty groups before this one.
__device__ __forceinline__ void write_segment(int* seg, int* rptr, int mode, int q, int b, int rb, int n, int u,
                                              int k, int sb, int pb, int mi, int s, int ne) {
  int p0, p1, r;
  if (mode == 2) {
    p0 = (int)(((long long)s * n) / k);
    p1 = (int)(((long long)(s + 1) * n) / k);
    r = sb + s;
  } else if (mode == 0) {
    p0 = 0; p1 = n; r = sb;
  } else {
    r = u / q + s;
    const int gs = max(u, r * q), ge = min(u + n, (r + 1) * q);
    p0 = gs - u; p1 = ge - u;
  }
  int* rec = seg + (size_t)(sb + s) * kSegWords;
  *reinterpret_cast<int4*>(rec) = make_int4(b, rb, p0, p1);
  *reinterpret_cast<int4*>(rec + 4) = make_int4(r, k > 1 ? pb + s : -1, k > 1 ? mi : -1, 0);
  if (mode != 1 || s > 0) {
    rptr[r] = sb + s;     // a cut: the segment starts its range
  } else {
    // the previous non-empty group's last page sits just before this group's gap
    const int r_prev = ne > 0 ? (u - kSegmentCostPages - 1) / q : -1;
    for (int rr = r_prev + 1; rr <= r; ++rr) rptr[rr] = sb;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a, char* ws) {
  int* hdr = reinterpret_cast<int*>(ws);
  int* grp = reinterpret_cast<int*>(ws + a.L.off_groups);
  int* seg = reinterpret_cast<int*>(ws + a.L.off_segments);
  int* rptr = reinterpret_cast<int*>(ws + a.L.off_range_ptr);
  int* mrg = reinterpret_cast<int*>(ws + a.L.off_merge);
  int* msync = reinterpret_cast<int*>(ws + a.L.off_merge_sync);
  __shared__ int sh[128];
  __shared__ int s_q, s_mode, s_U;
  // Where every group has a thread of its own its record stays in registers, and in shared
  // memory for the segments' pass.
  __shared__ int4 s_rec[2][kPlanThreads];
  int* s_sb = reinterpret_cast<int*>(s_rec);   // otherwise: the groups' first segments
  static_assert(sizeof(s_rec) >= kSmemGroups * sizeof(int), "room for either");
  const bool single = a.num_groups <= (int)blockDim.x;
  int4 rec0 = make_int4(0, 0, 0, 0), rec1 = rec0;   // (pages, pages before, segments, first segment), (first slot, merge record, line position, non-empty before)
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();

  // Sequence-length stamp (a wrapping sum, so order-free) and validation (the
  // smallest offending sequence is reported).
  unsigned hsum = 0;
  int errb = INT_MAX;
  for (int b = tid; b < a.B; b += blockDim.x) {
    const int S = a.seq_lens[b / a.seq_div];
    // query tokens of the sequence: T, or its tree's nodes (a count outside [0, T] is reported)
    const int n = a.tree && a.node_lens ? a.node_lens[b] : a.T;
    const uint32_t stamp = (uint32_t)S + (a.tree ? kNodeStamp * (uint32_t)n : 0u);
    hsum += mix32(stamp * 0x9E3779B1u + mix32((uint32_t)b + 0x632BE5ABu));
    if (S < 0 || S > a.max_rows || (S > 0 && S < n) || n < 0 || n > a.T) errb = min(errb, b);
  }

  // Pass A: pages per group and their exclusive prefix.
  int carry = 0, nonempty = 0, maxn = 0, nonempty_carry = 0;
  const int R = a.T * a.H;
  for (int base = 0; base < a.num_groups; base += blockDim.x) {
    const int g = base + tid;
    int n = 0;
    if (g < a.num_groups) {
      const int b = g / a.RB, rb = g % a.RB;
      int S = a.seq_lens[b / a.seq_div];
      S = S < 0 ? 0 : (S > a.max_rows ? a.max_rows : S);
      const int r_last = min(R, (rb + 1) * kRowsPerBlock) - 1;
      int vis = visible_limit(S, a.T, r_last / a.H, a.causal);
      // a group of rows past a tree's nodes needs no page
      if (a.tree && rb * kRowsPerBlock / a.H >= tree_nodes(a.node_lens, b, a.T, S)) vis = 0;
      n = (vis + kPage - 1) / kPage;
    }
    int v[3] = {n, n > 0 ? 1 : 0, 0}, tot[3];
    block_excl_scan3(v, tot, sh);
    if (g < a.num_groups) {
      const int ne = nonempty_carry + v[1];     // non-empty groups before g
      rec0.x = n;
      rec0.y = carry + v[0];
      rec1.z = carry + v[0] + kSegmentCostPages * ne;   // line position of its first page
      rec1.w = ne;
      if (!single) {
        grp[g * kGroupWords + 0] = rec0.x;
        grp[g * kGroupWords + 1] = rec0.y;
        grp[g * kGroupWords + 6] = rec1.z;
        grp[g * kGroupWords + 7] = rec1.w;
      }
      nonempty += n > 0;
      maxn = max(maxn, n);
    }
    carry += tot[0];
    nonempty_carry += tot[1];
  }
  block_reduce(hsum, errb, nonempty, maxn, sh);
  const int W = carry;
  if (tid == 0) {
    int q = (W + a.G - 1) / a.G;
    const int least = a.tree ? kTreeMinSplitPages : kMinSplitPages;
    q = q < least ? least : q;
    s_q = q;
    if (a.N > 0) s_mode = 2;
    else if (nonempty <= a.G && maxn <= (5 * q + 3) / 4) s_mode = 0;
    else s_mode = 1;
    if (s_mode == 1) {
      // balanced ranges over the line of pages and gaps
      const int U = W + kSegmentCostPages * (nonempty - 1);
      const int qw = (U + a.G - 1) / a.G;
      s_q = qw < least ? least : qw;
      s_U = U;
    }
  }
  __syncthreads();
  const int q = s_q, mode = s_mode;

  // Pass B: segments per group, segment/slot/merge bases; merge records.
  int cseg = 0, cpart = 0, cmrg = 0;
  for (int base = 0; base < a.num_groups; base += blockDim.x) {
    const int g = base + tid;
    int k = 0, n = 0;
    if (g < a.num_groups) {
      if (!single) {
        rec0 = *reinterpret_cast<const int4*>(grp + g * kGroupWords);
        rec1 = *reinterpret_cast<const int4*>(grp + g * kGroupWords + 4);
      }
      n = rec0.x;
      const int u = rec1.z;
      if (n > 0) {
        if (mode == 2) k = min(n, a.N);
        else if (mode == 0) k = 1;
        else k = (u + n - 1) / q - u / q + 1;
      }
    }
    const int part = k > 1 ? k : 0;
    const int mflag = (g < a.num_groups && k != 1) ? 1 : 0;
    int v[3] = {k, part, mflag}, tot[3];
    block_excl_scan3(v, tot, sh);
    if (g < a.num_groups) {
      const int sb = cseg + v[0];
      const int pb = part ? cpart + v[1] : -1;
      rec0.z = k;
      rec0.w = sb;
      rec1.x = pb;
      rec1.y = mflag ? cmrg + v[2] : -1;
      *reinterpret_cast<int4*>(grp + g * kGroupWords) = rec0;
      *reinterpret_cast<int4*>(grp + g * kGroupWords + 4) = rec1;
      if (single) {
        s_rec[0][g] = rec0;
        s_rec[1][g] = rec1;
      } else if (g < kSmemGroups) {
        s_sb[g] = sb;
      }
      msync[2 * g] = 0;       // merge record g's stored-partial count and merged-row count
      msync[2 * g + 1] = 0;
      if (mflag) {
        int* m = mrg + (size_t)(cmrg + v[2]) * kMergeWords;
        m[0] = g / a.RB; m[1] = g % a.RB; m[2] = (k > 1) ? pb : 0; m[3] = (k > 1) ? k : 0;
      }
    }
    cseg += tot[0]; cpart += tot[1]; cmrg += tot[2];
  }
  __syncthreads();
  const int total_seg = cseg;
  const int num_ranges = (mode == 1) ? (s_U + q - 1) / q : total_seg;

  // Pass C: segment records and range pointers, one segment per thread (its
  // group found by binary search over the segment bases), or one group per
  // thread when there are more groups than shared memory holds.
  if (a.num_groups <= kSmemGroups) {
    for (int i = tid; i < total_seg; i += blockDim.x) {
      int lo = 0, hi = a.num_groups;        // last group whose first segment is <= i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((single ? s_rec[0][mid].w : s_sb[mid]) <= i) lo = mid; else hi = mid;
      }
      const int g = lo;
      const int4 r0 = single ? s_rec[0][g] : *reinterpret_cast<const int4*>(grp + g * kGroupWords);
      const int4 r1 = single ? s_rec[1][g] : *reinterpret_cast<const int4*>(grp + g * kGroupWords + 4);
      write_segment(seg, rptr, mode, q, g / a.RB, g % a.RB, r0.x, r1.z, r0.z, r0.w, r1.x, r1.y, i - r0.w, r1.w);
    }
  } else {
    for (int g = tid; g < a.num_groups; g += blockDim.x) {
      const int* gr = grp + g * kGroupWords;
      const int k = gr[2];
      for (int s = 0; s < k; ++s)
        write_segment(seg, rptr, mode, q, g / a.RB, g % a.RB, gr[0], gr[6], k, gr[3], gr[4], gr[5], s, gr[7]);
    }
  }
  // Range pointers past the last range repeat the segment count, up to the
  // table's capacity: a decode CTA pair then reads its ranges' pointers
  // directly, without first reading the range count.
  for (int r = num_ranges + 1 + tid; r <= a.L.cap_ranges; r += blockDim.x) rptr[r] = total_seg;
  if (tid == 0) {
    rptr[num_ranges] = total_seg;
    hdr[MLA_HDR_B] = a.B; hdr[MLA_HDR_T] = a.T; hdr[MLA_HDR_H] = a.H; hdr[MLA_HDR_CAUSAL] = a.tree ? kPlanTree : a.causal;
    hdr[MLA_HDR_NUM_GROUPS] = a.num_groups;
    hdr[MLA_HDR_NUM_SEGMENTS] = total_seg;
    hdr[MLA_HDR_NUM_RANGES] = num_ranges;
    hdr[MLA_HDR_NUM_PARTIALS] = cpart;
    hdr[MLA_HDR_NUM_MERGE] = cmrg;
    hdr[MLA_HDR_SEQ_HASH] = (int)hsum;
    hdr[MLA_HDR_ERROR] = errb == INT_MAX ? 0 : MLA_ERR_DEVICE_CHECK;
    hdr[MLA_HDR_ERROR_INFO] = errb == INT_MAX ? 0 : errb;
    hdr[MLA_HDR_PAGES_PER_RANGE] = q;
    hdr[MLA_HDR_NUM_SLOTS] = a.G;
    hdr[MLA_HDR_OVERRIDE] = a.N;
    hdr[MLA_HDR_MAX_PAGES] = a.max_pages;
    hdr[MLA_HDR_OFF_SEGMENTS] = (int)a.L.off_segments;
    hdr[MLA_HDR_OFF_RANGE_PTR] = (int)a.L.off_range_ptr;
    hdr[MLA_HDR_OFF_MERGE] = (int)a.L.off_merge;
    hdr[MLA_HDR_OFF_PART_LSE] = (int)a.L.off_part_lse;
    hdr[MLA_HDR_OFF_PART_O] = (int)a.L.off_part_o;
    hdr[MLA_HDR_CAP_SEGMENTS] = a.L.cap_segments;
    hdr[MLA_HDR_CAP_PARTIALS] = a.L.cap_partials;
    hdr[MLA_HDR_CAP_RANGES] = a.L.cap_ranges;
    hdr[MLA_HDR_CAP_GROUPS] = a.L.cap_groups;
    hdr[MLA_HDR_MAGIC] = MLA_PLAN_MAGIC;
  }
}

// ------------------------------------------------------------------ batches that share prefixes
// Line positions ahead of a shared plan's group of so many query rows: what a segment more costs, in pages.
// Small segments change sooner (16 rows ~3.5 us, 32 ~5, 128 ~7, the partial states' stores among it; a page
// 0.87).  Plan and decode of samples of a prompt (own groups of 16 rows), documents (32) and 40 FP8 sequences (128
// and 64) in us: 8 for all 38.1, 104, 74.4; 4 for all 36.6, 119, 75.8; 4 + rows / 32 35.4, 109, 75.6; this 34.5, 103,
// 74.6.  (On those three batches; on no others.)  The plan itself takes 5.4 to 6.2 us, a chain of dependent loads and block scans (10 behind a decode that
// has emptied the L2 of its code).
__device__ __forceinline__ int shared_gap(int rows) { return min(2 + rows / 8, 8); }
// Sharing a set's pages costs a segment per 128 of its rows and the partial states of all of
// them, twice, stored and merged, which gets dearer as they fill the L2.  In pages, by the decode with
// and without (one set, 76 pairs; us):
//   8 x 16 heads, prefix 512: 16.5 and 15.9; 1536: 17.4 and 17.9; 4096: 19.5 and 21.9
//   96 x 16 heads, prefix 512: 29.1 and 31.2; 1536: 32.2 and 50.8; 12000: 55 and 249
//   48 x 64 heads, prefix 512: 27.6 and 25.8; 1536: 31.5 and 36.2; 12000: 80 and 127
//   96 x 3 tokens x 64 heads, prefix 4096: 208 and 171; 48 of those, 4096: 104 and 95; 12000: 215 and 219
// Of 79 such batches (4 to 96 sequences, prefixes of 512 to 12000) the rule takes the faster way, or one that is
// within 5 % of it (kSharedGroupCost, kSharedRowsPerPage).
constexpr int kSharedLeastSaved = 1;                             // pages per range, over all sets

struct SharedPlanArgs {
  const int32_t *seq_lens, *q_lens;
  int B, T, H, causal, G, N, max_pages, RB, num_sets;
  const int32_t *set_ptr, *prefix_lens;
  WsLayout L;
};

// The block's sum of one non-negative int per thread, ending at 2^30.
__device__ int block_sum_to(int v, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  constexpr int kEnd = 1 << 30;
  v = min(v, kEnd);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = min(v + __shfl_xor_sync(0xffffffffu, v, o), kEnd);
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  int s = lane < nwarps ? sh[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s = min(s + __shfl_xor_sync(0xffffffffu, s, o), kEnd);
  __syncthreads();
  return s;
}

// The set of sequence b: the last p with ptr[p] <= b, if b < ptr[p + 1]; else -1.
__device__ __forceinline__ int set_of(const int* ptr, int num_sets, int b) {
  int lo = 0, hi = num_sets + 1;      // ptr[lo] <= b < ptr[hi], where there are such
  if (num_sets == 0 || b < ptr[0] || b >= ptr[num_sets]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ptr[mid] <= b) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_shared_kernel(SharedPlanArgs a, char* ws) {
  int* hdr = reinterpret_cast<int*>(ws);
  int* grp = reinterpret_cast<int*>(ws + a.L.off_groups);
  int* seg = reinterpret_cast<int*>(ws + a.L.off_segments);
  int* rptr = reinterpret_cast<int*>(ws + a.L.off_range_ptr);
  int* mrg = reinterpret_cast<int*>(ws + a.L.off_merge);
  int* msync = reinterpret_cast<int*>(ws + a.L.off_merge_sync);
  extern __shared__ int dyn[];
  const int P = a.num_sets;
  int* s_ptr = dyn;                   // [P + 1]
  int* s_base = s_ptr + P + 1;        // [P + 1]: the sets' first groups
  int* s_pages = s_base + P + 1;      // [P]: shared pages; at first the rows that every live member sees
  int* s_first = s_pages + P;         // [P]: the first live member
  int* s_live = s_first + P;          // [P]: how many are
  __shared__ int sh[128];
  __shared__ int s_q, s_mode, s_U, s_gap;      // s_gap: ahead of the first group, which needs none
  const int tid = threadIdx.x;
  const int R = a.T * a.H;
  pdl_wait();
  pdl_trigger();

  // (a thread's first sequence is asked for together with the sets)
  int S_first = 0, n_first = a.T;
  if (tid < a.B) {
    S_first = a.seq_lens[tid];
    if (a.q_lens) n_first = a.q_lens[tid];
  }
  // The sets; bounds that do not rise, or pass the batch, are reported and nothing is shared.
  bool bad_set = false;
  for (int p = tid; P > 0 && p <= P; p += blockDim.x) {
    const int v = a.set_ptr[p];
    bad_set = bad_set || v < 0 || v > a.B || (p < P && a.set_ptr[p + 1] < v);
    s_ptr[p] = v;
    if (p < P) {
      bad_set = bad_set || a.prefix_lens[p] < 0;
      s_pages[p] = INT_MAX;
      s_first[p] = INT_MAX;
      s_live[p] = 0;
    }
  }
  const int sets = __syncthreads_or(bad_set) ? 0 : P;

  // Lengths: the stamp, what is wrong with them, and what the sets' members see.
  unsigned hsum = 0;
  int errb = INT_MAX;
  const int max_rows = a.max_pages * kPage;
  for (int b = tid; b < a.B; b += blockDim.x) {
    const int S = b == tid ? S_first : a.seq_lens[b], n = b == tid ? n_first : a.q_lens ? a.q_lens[b] : a.T;
    hsum += mix32(((uint32_t)S + kNodeStamp * (uint32_t)n) * 0x9E3779B1u + mix32((uint32_t)b + 0x632BE5ABu));
    if (S < 0 || S > max_rows || (S > 0 && S < n) || n < 0 || n > a.T) errb = min(errb, b);
    const int rows = S < 0 ? 0 : min(S, max_rows);
    const int p = set_of(s_ptr, sets, b);
    if (p >= 0 && rows > 0) {
      // its first token sees the fewest rows (a sequence without tokens: no bound but its length)
      const int q = tree_nodes(a.q_lens, b, a.T, rows);
      atomicMin(&s_pages[p], min(rows, visible_limit(rows, q, 0, a.causal)));
      atomicMin(&s_first[p], b);
      atomicAdd(&s_live[p], 1);
    }
  }
  __syncthreads();

  // What each set shares: whole pages, and only where that pays (the workspace is laid out for what can).
  int saved_all = 0;
  for (int p = tid; p < P; p += blockDim.x) {
    int pages = 0;
    if (sets > 0 && s_pages[p] != INT_MAX && may_share(R, a.max_pages)) {
      const long long members = s_ptr[p + 1] - s_ptr[p], rows = members * R;
      const long long groups = (rows + kRowsPerBlock - 1) / kRowsPerBlock;
      pages = min(s_pages[p], a.prefix_lens[p]) / kPage;
      const long long saved = ((long long)s_live[p] * a.RB - groups) * pages - (kSharedGroupCost + rows / kSharedRowsPerPage) * groups;
      if (saved <= 0) pages = 0;
      else saved_all = (int)min((long long)saved_all + saved, 1LL << 24);
    }
    s_pages[p] = pages;
  }
  // (the sum over the threads, as far as it matters)
  const bool pays = block_sum_to(saved_all, sh) > kSharedLeastSaved * a.G;
  int prefix_groups = 0;
  for (int base = 0; base < P; base += blockDim.x) {
    const int p = base + tid;
    int count = 0;
    if (p < P) {
      if (!pays) s_pages[p] = 0;
      if (s_pages[p] > 0) count = (int)(((long long)(s_ptr[p + 1] - s_ptr[p]) * R + kRowsPerBlock - 1) / kRowsPerBlock);
    }
    int v[3] = {count, 0, 0}, tot[3];
    block_excl_scan3(v, tot, sh);
    if (p < P) s_base[p] = prefix_groups + v[0];
    prefix_groups += tot[0];
  }
  if (tid == 0) s_base[P] = prefix_groups;
  __syncthreads();
  const int num_groups = prefix_groups + a.B * a.RB;

  // Pass A: the groups' pages and rows, and their places on the line.  (Where every group has a
  // thread its record stays in registers.)
  const bool single = num_groups <= (int)blockDim.x;
  int4 r0 = make_int4(0, 0, 0, 0), r1 = r0, r2 = r0;
  int carry = 0, nonempty = 0, maxn = 0, ne_carry = 0, gaps = 0;
  for (int base = 0; base < num_groups; base += blockDim.x) {
    const int g = base + tid;
    int n = 0, page0 = 0, table = 0, row0 = 0, rows = 0, flag = 0;
    if (g < prefix_groups) {
      int lo = 0, hi = P;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_base[mid] <= g) lo = mid; else hi = mid;
      }
      const int first = (g - s_base[lo]) * kRowsPerBlock;
      n = s_pages[lo];
      table = s_first[lo];
      row0 = s_ptr[lo] * R + first;
      rows = min(kRowsPerBlock, (s_ptr[lo + 1] - s_ptr[lo]) * R - first);
      flag = 1 << 16;
    } else if (g < num_groups) {
      const int b = (g - prefix_groups) / a.RB, first = (g - prefix_groups) % a.RB * kRowsPerBlock;
      int S = a.seq_lens[b];
      S = S < 0 ? 0 : min(S, max_rows);
      const int q = tree_nodes(a.q_lens, b, a.T, S);
      rows = min(kRowsPerBlock, R - first);
      table = b;
      row0 = b * R + first;
      const int p = set_of(s_ptr, sets, b);
      const int last = min(q - 1, (first + rows - 1) / a.H);      // the last token of the group's rows
      const int seen = first / a.H < q ? visible_limit(S, q, last, a.causal) : 0;
      page0 = p >= 0 ? s_pages[p] : 0;
      n = max(0, (seen + kPage - 1) / kPage - page0);
    }
    const int gap = n > 0 ? shared_gap(rows) : 0;
    int v[3] = {n, n > 0 ? 1 : 0, gap}, tot[3];
    block_excl_scan3(v, tot, sh);
    if (g < num_groups) {
      int4* rec = reinterpret_cast<int4*>(grp + (size_t)g * kSharedGroupWords);
      const int ne = ne_carry + v[1];
      if (n > 0 && ne == 0) s_gap = gap;
      r0 = make_int4(n, page0, 0, 0);
      r1 = make_int4(-1, table, row0, rows | flag);
      r2 = make_int4(carry + v[0] + gaps + v[2] + gap, ne, gap, 0);       // (the first group's gap is taken off below)
      if (!single) {
        rec[0] = r0;
        rec[1] = r1;
      }
      rec[2] = r2;
      nonempty += n > 0;
      maxn = max(maxn, n);
    }
    carry += tot[0];
    ne_carry += tot[1];
    gaps += tot[2];
  }
  block_reduce(hsum, errb, nonempty, maxn, sh);
  if (tid == 0) {
    int q = (carry + a.G - 1) / a.G;
    q = q < kTreeMinSplitPages ? kTreeMinSplitPages : q;
    s_q = q;
    s_mode = a.N > 0 ? 2 : nonempty <= a.G && maxn <= (5 * q + 3) / 4 ? 0 : 1;
    if (s_mode == 1) {
      const int U = carry + gaps - s_gap;
      const int qw = (U + a.G - 1) / a.G;
      s_q = qw < kTreeMinSplitPages ? kTreeMinSplitPages : qw;
      s_U = U;
    }
  }
  __syncthreads();
  const int q = s_q, mode = s_mode;

  // Pass B: segments and partial rows of each group, merge records, the segments.  A group
  // writes final rows where nothing is to be merged with them.
  int cseg = 0, crow = 0, cmrg = 0;
  for (int base = 0; base < num_groups; base += blockDim.x) {
    const int g = base + tid;
    int k = 0, part = 0, merged = 0;
    const bool own = g >= prefix_groups;
    if (g < num_groups) {
      if (!single) {
        const int4* rec = reinterpret_cast<const int4*>(grp + (size_t)g * kSharedGroupWords);
        r0 = rec[0]; r1 = rec[1]; r2 = rec[2];
      }
      const int n = r0.x, u = r2.x - s_gap;
      if (n > 0) k = mode == 2 ? min(n, a.N) : mode == 0 ? 1 : (u + n - 1) / q - u / q + 1;
      const bool shares = own && r0.y > 0;
      part = k > 0 && (k > 1 || shares || !own) ? k * (r1.w & 0xFFFF) : 0;
      merged = own && (k != 1 || shares) ? 1 : 0;
    }
    int v[3] = {k, part, merged}, tot[3];
    block_excl_scan3(v, tot, sh);
    if (g < num_groups) {
      const int sb = cseg + v[0], first_row = part > 0 ? crow + v[1] : -1;
      int4* rec = reinterpret_cast<int4*>(grp + (size_t)g * kSharedGroupWords);
      rec[0] = make_int4(r0.x, r0.y, k, sb);
      rec[1] = make_int4(first_row, r1.y, r1.z, r1.w);
      msync[2 * g] = 0;
      msync[2 * g + 1] = 0;
      if (merged) {
        const int b = r1.y, p = r0.y > 0 ? set_of(s_ptr, sets, b) : -1;
        const int in_set = p >= 0 ? r1.z - s_ptr[p] * R : 0;     // its first row among the set's
        int4* m = reinterpret_cast<int4*>(mrg + (size_t)(cmrg + v[2]) * kSharedMergeWords);
        m[0] = make_int4(r1.z, r1.w & 0xFFFF, g, p >= 0 ? s_base[p] + in_set / kRowsPerBlock : -1);
        m[1] = make_int4(in_set % kRowsPerBlock, 0, 0, 0);
      }
      // line position of the group's first page: the ranges between the group before and this one are empty
      const int n = r0.x, u = r2.x - s_gap;
      for (int s = 0; s < k; ++s) {
        int p0, p1, r;
        if (mode == 2) {
          p0 = (int)((long long)s * n / k);
          p1 = (int)((long long)(s + 1) * n / k);
          r = sb + s;
        } else if (mode == 0) {
          p0 = 0; p1 = n; r = sb;
        } else {
          r = u / q + s;
          p0 = max(u, r * q) - u;
          p1 = min(u + n, (r + 1) * q) - u;
        }
        int4* out = reinterpret_cast<int4*>(seg + (size_t)(sb + s) * kSegWords);
        out[0] = make_int4(r1.y, r1.z, r0.y + p0, r0.y + p1);
        out[1] = make_int4(r, first_row < 0 ? -1 : first_row + s * (r1.w & 0xFFFF), g, r1.w);
        if (mode != 1 || s > 0) {
          rptr[r] = sb + s;
        } else {
          const int r_prev = r2.y > 0 ? (u - r2.z - 1) / q : -1;
          for (int rr = r_prev + 1; rr <= r; ++rr) rptr[rr] = sb;
        }
      }
    }
    cseg += tot[0]; crow += tot[1]; cmrg += tot[2];
  }
  const int num_ranges = mode == 1 ? (s_U + q - 1) / q : cseg;
  for (int r = num_ranges + 1 + tid; r <= a.L.cap_ranges; r += blockDim.x) rptr[r] = cseg;
  if (tid == 0) {
    rptr[num_ranges] = cseg;
    hdr[MLA_HDR_B] = a.B; hdr[MLA_HDR_T] = a.T; hdr[MLA_HDR_H] = a.H; hdr[MLA_HDR_CAUSAL] = kPlanShared + a.causal;
    hdr[MLA_HDR_NUM_GROUPS] = num_groups;
    hdr[MLA_HDR_NUM_SEGMENTS] = cseg;
    hdr[MLA_HDR_NUM_RANGES] = num_ranges;
    hdr[MLA_HDR_NUM_PARTIALS] = crow;
    hdr[MLA_HDR_NUM_MERGE] = cmrg;
    hdr[MLA_HDR_SEQ_HASH] = (int)hsum;
    // (sequence B stands for the sets)
    const int info = errb != INT_MAX ? errb : a.B;
    const bool bad = errb != INT_MAX || sets != P;
    hdr[MLA_HDR_ERROR] = bad ? MLA_ERR_DEVICE_CHECK : 0;
    hdr[MLA_HDR_ERROR_INFO] = bad ? info : 0;
    hdr[MLA_HDR_PAGES_PER_RANGE] = q;
    hdr[MLA_HDR_NUM_SLOTS] = a.G;
    hdr[MLA_HDR_OVERRIDE] = a.N;
    hdr[MLA_HDR_MAX_PAGES] = a.max_pages;
    hdr[MLA_HDR_OFF_SEGMENTS] = (int)a.L.off_segments;
    hdr[MLA_HDR_OFF_RANGE_PTR] = (int)a.L.off_range_ptr;
    hdr[MLA_HDR_OFF_MERGE] = (int)a.L.off_merge;
    hdr[MLA_HDR_OFF_PART_LSE] = (int)a.L.off_part_lse;
    hdr[MLA_HDR_OFF_PART_O] = (int)a.L.off_part_o;
    hdr[MLA_HDR_CAP_SEGMENTS] = a.L.cap_segments;
    hdr[MLA_HDR_CAP_PARTIALS] = a.L.cap_partials;
    hdr[MLA_HDR_CAP_RANGES] = a.L.cap_ranges;
    hdr[MLA_HDR_CAP_GROUPS] = a.L.cap_groups;
    hdr[MLA_HDR_MAGIC] = MLA_PLAN_MAGIC;
  }
}

}  // namespace

cudaError_t launch_plan_shared(const int32_t* seq_lens, const SharedQueries& q, const SharedSets& sets,
                               const mla_geom* g, const mla_batch* b, const WsLayout& L, void* ws, cudaStream_t st) {
  SharedPlanArgs a{seq_lens, q.q_lens, b->B, b->T, g->H, b->causal ? 1 : 0, L.num_slots, b->num_splits_override,
                   b->max_pages, (b->T * g->H + kRowsPerBlock - 1) / kRowsPerBlock, sets.count, sets.ptr,
                   sets.prefix_lens, L};
  const size_t smem = (5 * (size_t)sets.count + 2) * sizeof(int);
  // (more than 48 KB has to be asked for; as often as it comes, it is the same)
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(plan_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (5 * kMaxSharedSequences + 2) * (int)sizeof(int)) != cudaSuccess)
    return cudaErrorInvalidValue;
  // as many threads as groups, at most, for cheap barriers
  int threads = kTreePlanThreads;
  while (threads < kPlanThreads && threads < L.cap_groups) threads *= 2;
  return launch_pdl(plan_shared_kernel, dim3(1), dim3(threads), smem, st, a, reinterpret_cast<char*>(ws));
}

cudaError_t launch_plan(const int32_t* seq_lens, const mla_geom* g, const mla_batch* b, const WsLayout& L,
                        void* ws, cudaStream_t st, int seq_div, int max_rows, const TreeNodes* tree) {
  PlanArgs a;
  a.seq_lens = seq_lens;
  a.seq_div = seq_div;
  a.B = b->B; a.T = b->T; a.H = g->H; a.causal = b->causal ? 1 : 0;
  a.G = L.num_slots; a.N = b->num_splits_override; a.max_pages = b->max_pages;
  a.max_rows = max_rows > 0 ? max_rows : b->max_pages * kPage;
  a.RB = (b->T * g->H + kRowsPerBlock - 1) / kRowsPerBlock;
  a.num_groups = b->B * a.RB;
  a.tree = tree != nullptr;
  a.node_lens = tree ? tree->node_lens : nullptr;
  a.L = L;
  int threads = kPlanThreads;
  if (tree)
    for (threads = kTreePlanThreads; threads < kPlanThreads && threads < a.num_groups + a.num_groups / 4;) threads *= 2;
  return launch_pdl(plan_kernel, dim3(1), dim3(threads), 0, st, a, reinterpret_cast<char*>(ws));
}

}  // namespace mla
