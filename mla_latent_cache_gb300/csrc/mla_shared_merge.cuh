// The merge of a shared plan's partial states, run by the decode kernel's own CTAs: a
// query row's parts are those of its sequence's own pages and those of the pages that its
// set shares, which 128 rows of several sequences computed together.
//
// The formula and the counters are mla_plan_merge.cuh's: o = sum of w_r o_r / sum of w_r, w_r =
// exp(lse_r - max), all in fp32.  The parts lie in two places.  A merge record stands for up to 128
// rows of a sequence; its rows lie in one or two groups of the set (128 rows each, whatever the
// sequence).  Partial states take as many rows as their group has, not 128: a sequence's
// own group at 16 heads has 16.
//
// Bound by latency: it begins when the last partial state is stored, and nothing else is left to do.
// From there to the end, 64 sequences x 128 heads (45 rows of two parts, 180 KB, a CTA) 14 -> 8 us (HBM
// alone 5), 40 FP8 sequences x 64 heads x 3 tokens 10 -> 7 us, 48 requests x 32 heads about a document of 32768 rows 11 -> 6 us, with records
// looked up ahead, all parts on their way at once, and one thread for a row's weights.
#pragma once

#include "mla_plan_merge.cuh"

namespace mla {
namespace merge {

// Where a group's partial states are: part r of the group's row i at base + r * rows + i.
struct Parts {
  int group, k, base, rows;
};
__device__ __forceinline__ Parts parts_of(const int* grp, int g) {
  const int* rec = grp + (size_t)g * kSharedGroupWords;
  const int k = __ldcg(rec + 2), base = __ldcg(rec + 4), rows = __ldcg(rec + 7);
  return {g, base < 0 ? 0 : k, base, rows & 0xFFFF};
}

struct RowParts {
  Parts own, set0, set1;    // set1: the set's next group (k = 0 where the rows end before it)
  int first_row, rows, place;
  bool foreign;             // the sequence does not hold the set's pages: the set's parts are not its own
  // The partial row of part r of the record's row i, or -1.
  __device__ __forceinline__ long long at(int i, int r) const {
    if (r < own.k) return own.base + (long long)r * own.rows + i;
    const int j = r - own.k, p = place + i;
    const bool next = p >= kRowsPerBlock;
    const int k = next ? set1.k : set0.k;
    if (j >= k || foreign) return -1;
    return next ? set1.base + (long long)j * set1.rows + (p - kRowsPerBlock) : set0.base + (long long)j * set0.rows + p;
  }
  __device__ __forceinline__ int most() const { return own.k + max(set0.k, set1.k); }
};

// The records of a share, as many as are looked up at once.
constexpr int kRecords = 8;
struct Share {
  RowParts p;
  int row_a, row_b;          // this CTA's rows of the record
};

__device__ __forceinline__ void copy16(float* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// Where the parts wait in shared memory: as many as the attention leaves room for, a row's one after
// the other.  Their rows, and their log-sum-exps, then weights; the rows' places in the output.
constexpr int kStaged = 108;
struct Staged {
  alignas(16) float o[kStaged][kDLat];
  int part[kStaged];
  float weight[kStaged];
  int row[kStaged];
};

// Slots [slot, slot + nslots) of the records (per_rec each), `most` parts to a row at most, nslots * most <= kStaged.
// All parts are on their way at once, and what goes for a whole row is done by one thread: with four
// columns to a thread, and the weights worked out by each of 128, a row took 0.7 us.
template <int G>
__device__ __forceinline__ void merge_shared_rows(const Out& a, const float* part_o, const float* part_lse,
                                                  const Share* shares, int per_rec, int slot, int nslots, int most, Staged& st) {
  static_assert(kStaged <= G * 128 && kDLat == 512, "a thread to a part, 128 to its values");
  const int tid = threadIdx.x, n = nslots * most;
  float lse = -INFINITY;
  if (tid < n) {
    const int s = tid / most, r = tid - s * most, i = (slot + s) / per_rec, row = slot + s - i * per_rec;
    const bool in = row < shares[i].p.rows;
    const long long pr = in ? shares[i].p.at(row, r) : -1;
    if (pr >= 0) lse = __ldcg(part_lse + pr);
    st.part[tid] = (int)pr;
    if (r == 0) st.row[s] = in ? shares[i].p.first_row + row : -1;
  }
  __syncthreads();
#pragma unroll 2
  for (int k = tid / 128; k < n; k += G) {
    const int pr = st.part[k];
    if (pr >= 0) copy16(&st.o[k][tid % 128 * 4], part_o + (size_t)pr * kDLat + tid % 128 * 4);
  }
  if (tid < n) st.weight[tid] = lse;
  __syncthreads();
  if (tid < nslots && st.row[tid] >= 0) {
    float* const w = st.weight + tid * most;
    float mx = -INFINITY, l = 0.f;
    for (int r = 0; r < most; ++r) mx = fmaxf(mx, w[r]);
    for (int r = 0; r < most; ++r) {
      w[r] = w[r] == -INFINITY ? 0.f : __expf(w[r] - mx);
      l += w[r];
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int r = 0; r < most; ++r) w[r] *= inv;
    a.lse[st.row[tid]] = l > 0.f ? mx + logf(l) : -INFINITY;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const int c = tid % 64 * 8;
#pragma unroll 1
  for (int s = tid / 64; s < nslots; s += 2 * G) {
    const int row = st.row[s];
    if (row < 0) continue;
    float sum[8] = {};
#pragma unroll 2
    for (int k = s * most; k < (s + 1) * most; ++k) {
      const float w = st.weight[k];
      if (w == 0.f) continue;            // (no part, or an empty one: its values are anything)
      const float4 x = *reinterpret_cast<const float4*>(&st.o[k][c]), y = *reinterpret_cast<const float4*>(&st.o[k][c + 4]);
      sum[0] = fmaf(w, x.x, sum[0]); sum[1] = fmaf(w, x.y, sum[1]); sum[2] = fmaf(w, x.z, sum[2]); sum[3] = fmaf(w, x.w, sum[3]);
      sum[4] = fmaf(w, y.x, sum[4]); sum[5] = fmaf(w, y.y, sum[5]); sum[6] = fmaf(w, y.z, sum[6]); sum[7] = fmaf(w, y.w, sum[7]);
    }
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(sum[2 * j], sum[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(a.o_lat + (size_t)row * kDLat + c) = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __syncthreads();   // the parts are read: others may come in their place
}

// One row, its parts split over the G groups of threads (all of the CTA).
template <int G>
__device__ __forceinline__ void merge_shared_row(const Out& a, const float* part_o, const float* part_lse,
                                                 const RowParts& p, int row, float* s_st, int grp, int t) {
  const int c = 4 * t;
  State st{-INFINITY, 0.f, 0.f, 0.f, 0.f, 0.f};
  const Parts& set_of = p.place + row < kRowsPerBlock ? p.set0 : p.set1;
  if (p.own.k > 0) {
    const size_t r0 = p.at(row, 0);
    fold_partials(st, part_o + r0 * kDLat + c, part_lse + r0, (size_t)p.own.rows * kDLat, p.own.rows, grp, G, p.own.k);
  }
  if (set_of.k > 0 && !p.foreign) {
    const size_t r0 = p.at(row, p.own.k);
    fold_partials(st, part_o + r0 * kDLat + c, part_lse + r0, (size_t)set_of.rows * kDLat, set_of.rows, grp, G, set_of.k);
  }
  float* my = s_st + (grp * 6) * 128 + t;
  my[0] = st.m; my[128] = st.l; my[256] = st.a0; my[384] = st.a1; my[512] = st.a2; my[640] = st.a3;
  __syncthreads();
  if (grp == 0) {
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < G; ++j) mx = fmaxf(mx, s_st[(j * 6) * 128 + t]);
    State m{mx, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (mx != -INFINITY) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const float* sj = s_st + (j * 6) * 128 + t;
        const float f = sj[0] == -INFINITY ? 0.f : __expf(sj[0] - mx);
        m.l = fmaf(f, sj[128], m.l);
        m.a0 = fmaf(f, sj[256], m.a0);
        m.a1 = fmaf(f, sj[384], m.a1);
        m.a2 = fmaf(f, sj[512], m.a2);
        m.a3 = fmaf(f, sj[640], m.a3);
      }
    }
    store_row(a, (size_t)p.first_row + row, c, m);
  }
  __syncthreads();
}

// Bounded wait until a group's partial rows are all stored; false (after recording MLA_ERR_TIMEOUT) if
// its count never completes.
__device__ __forceinline__ bool wait_parts(int* hdr, const int* msync, const Parts& p) {
  const long long t0 = clock64();
  while (p.k > 0) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(msync + 2 * p.group) : "memory");
    if (v >= kCountsPerSegment * p.k) break;
    if (clock64() - t0 > MLA_PIPELINE_WAIT_LIMIT) {
      record_error(hdr, MLA_ERR_TIMEOUT, 61);
      return false;
    }
    __nanosleep(64);
  }
  return true;
}

// n rows of a group are merged; the CTA that merges its last ones zeroes its counters.
__device__ __forceinline__ void count_merged(int* msync, const Parts& p, int n) {
  if (n <= 0 || p.k == 0) return;
  if (atomicAdd(msync + 2 * p.group + 1, n) + n == p.rows) {
    atomicExch(msync + 2 * p.group, 0);
    atomicExch(msync + 2 * p.group + 1, 0);
  }
}

// The rows of a CTA's share of the merge: slots [first, end) of num_merge records, per_rec slots each.
struct Slots {
  int per_rec;
  long long first, end;
  __device__ __forceinline__ Slots(int num_merge, int R, int cta, int nctas) : per_rec(min(R, kRowsPerBlock)) {
    const long long V = (long long)num_merge * per_rec, per = (V + nctas - 1) / nctas;
    first = cta * per;
    end = min(V, first + per);
  }
  // The slots from v on that are looked up at once: of the record of v and up to kRecords - 1 more.
  __device__ __forceinline__ long long record(long long v) const { return v / per_rec; }
  __device__ __forceinline__ int count(long long v) const { return (int)(min(end, (record(v) + kRecords) * per_rec) - v); }
};

// What tells whether the sequences of a set hold the same pages.
struct Tables {
  const int32_t* block_table;
  int stride;
  const int32_t *seq_lens, *q_lens;
  int T, R, max_rows, checked;
};
// Whether sequence b, which has query tokens, holds other blocks than table row `read` in its first `pages`
// pages.  Forks share leading pages, so that the last page tells; checked, all are compared.
__device__ __forceinline__ bool holds_others(const Tables& t, int b, int read, int pages) {
  const int S = t.seq_lens[b];
  if (b == read || tree_nodes(t.q_lens, b, t.T, S < 0 ? 0 : min(S, t.max_rows)) == 0) return false;
  const int32_t* const mine = t.block_table + (size_t)b * t.stride;
  const int32_t* const his = t.block_table + (size_t)read * t.stride;
  bool others = mine[pages - 1] != his[pages - 1];
  for (int p = 0; t.checked && p < pages - 1; ++p) others = others || mine[p] != his[p];
  return others;
}

// The records of the slots from v on, and their groups, to shares[]: one warp, four lanes to a record.
// A sequence that does not hold the pages of its set is reported, and gets none of the set's parts: what
// was attended there are somebody else's rows.  (Looked at here, while the pages are attended: by
// the softmax warps, at each segment, it cost documents 105 -> 117 us.)
__device__ __forceinline__ void look_up(Share* shares, char* ws, const WsLayout& L, const Slots& slots, long long v,
                                        const Tables& tables) {
  const int* grps = reinterpret_cast<const int*>(ws + L.off_groups);
  const int* mrg = reinterpret_cast<const int*>(ws + L.off_merge);
  const int i = (threadIdx.x & 31) / 4, which = threadIdx.x % 4;
  const long long i0 = slots.record(v);
  const int slot = (int)(v - i0 * slots.per_rec), nslots = slots.count(v);
  if (i * slots.per_rec >= slot + nslots) return;
  const int* rec = mrg + (size_t)(i0 + i) * kSharedMergeWords;
  const int first_row = __ldcg(rec + 0), rows = __ldcg(rec + 1), own = __ldcg(rec + 2), set = __ldcg(rec + 3),
            place = __ldcg(rec + 4);
  Share& s = shares[i];
  if (which == 3) {
    s.p.first_row = first_row;
    s.p.rows = rows;
    s.p.place = place;
    const int b = first_row / tables.R;
    s.p.foreign = set >= 0 && holds_others(tables, b, __ldcg(grps + (size_t)set * kSharedGroupWords + 5),
                                           __ldcg(grps + (size_t)own * kSharedGroupWords + 1));
    if (s.p.foreign) record_error(reinterpret_cast<int*>(ws), MLA_ERR_DEVICE_CHECK, b);
    s.row_a = i == 0 ? slot : 0;
    s.row_b = min(rows, slot + nslots - i * slots.per_rec);
  } else {
    const int g = which == 0 ? own : set < 0 || (which == 2 && place + rows <= kRowsPerBlock) ? -1 : set + which - 1;
    (which == 0 ? s.p.own : which == 1 ? s.p.set0 : s.p.set1) = g >= 0 ? parts_of(grps, g) : Parts{0, 0, 0, 0};
  }
}

// CTA `cta` of `nctas` merges its share of the plan's rows; arguments as for merge_plan_share.
// Up to kRecords records are looked up and waited for at once and their rows merged in common; the
// first ones were looked up while the pages were attended (shares[]).  One after another, each with its
// chain of record, groups, counters and states, they took 11 us after the last page of 48 x 128 rows of
// two to three parts each.
template <int G>
__device__ __forceinline__ void merge_shared_share(const Out& a, char* ws, const WsLayout& L, int num_merge, int cta,
                                                   int nctas, float* s_st, Share* shares, Staged& st, const Tables& tables) {
  int* hdr = reinterpret_cast<int*>(ws);
  int* msync = reinterpret_cast<int*>(ws + L.off_merge_sync);
  const float* part_lse = reinterpret_cast<const float*>(ws + L.off_part_lse);
  const float* part_o = reinterpret_cast<const float*>(ws + L.off_part_o);
  const Slots slots(num_merge, a.T * a.H, cta, nctas);
  const int grp = threadIdx.x / (kDLat / 4);
  const int t = threadIdx.x % (kDLat / 4);
  for (long long v = slots.first; v < slots.end;) {
    if (v > slots.first) {
      if (threadIdx.x < 32) look_up(shares, ws, L, slots, v, tables);
      __syncthreads();
    }
    const int slot = (int)(v - slots.record(v) * slots.per_rec), nslots = slots.count(v);
    const int records = (slot + nslots + slots.per_rec - 1) / slots.per_rec;
    // Four threads to a record.  The set's groups are waited for where this CTA's rows lie in them: rows
    // before `cut` are in the first.
    const int i = threadIdx.x / 4, which = threadIdx.x % 4;
    Parts mine{0, 0, 0, 0};
    int merged = 0;
    bool ok = true;
    if (i < records && which < 3) {
      const Share& s = shares[i];
      mine = which == 0 ? s.p.own : which == 1 ? s.p.set0 : s.p.set1;
      const int cut = min(max(kRowsPerBlock - s.p.place, s.row_a), s.row_b);
      merged = s.row_a >= s.row_b ? 0 : which == 0 ? s.row_b - s.row_a : which == 1 ? cut - s.row_a : s.row_b - cut;
      if (merged > 0) ok = wait_parts(hdr, msync, mine);
    }
    if (!__syncthreads_and(ok)) return;
    int most = 0;
    for (int j = 0; j < records; ++j) most = max(most, shares[j].p.most());
    if (most <= kStaged) {
      const int batch = kStaged / max(most, 1);
      for (int s = 0; s < nslots; s += batch)
        merge_shared_rows<G>(a, part_o, part_lse, shares, slots.per_rec, slot + s, min(batch, nslots - s), max(most, 1), st);
    } else {
      for (int j = 0; j < records; ++j)
        for (int row = shares[j].row_a; row < shares[j].row_b; ++row)
          merge_shared_row<G>(a, part_o, part_lse, shares[j].p, row, s_st, grp, t);
    }
    __syncthreads();   // this CTA's reads of those rows are done
    count_merged(msync, mine, merged);
    v += nslots;
  }
}

}  // namespace merge
}  // namespace mla
