// Verification of drafted tokens (a tree, or a chain as a tree without branches)
// against the target's probabilities, from given random numbers.
//
// Rule, per sequence.  Node 0 is the last token already decided; node t > 0 holds a
// drafted token and hangs on parents[t] < t.  Let cur be the last accepted node (0 at
// first), p the target's probabilities after cur, q the drafter's there.  The children x
// of cur are tried in index order; after k of them were refused, what is left of p is
// R_k = max(p - C_k q, 0) with mass Z_k, where C_0 = 0, Z_0 = 1, C_{k+1} = C_k + Z_k and
// Z_k = sum R_k.  Child x is accepted when R_k(x) > 0 and u q(x) Z_k < R_k(x), and
// becomes cur; when no child is left, the last token is drawn from R_k.
//   This is rejection sampling with a chain of residuals: accept with probability
//   min(1, r_k(x) / q(x)), r_k = R_k / Z_k, and r_{k+1} is max(r_k - q, 0) normalised.
//   Z_k max(r_k - q, 0) = max(R_k - Z_k q, 0), and a value that has reached 0 stays
//   there, so R_{k+1} = max(p - (Z_0 + ... + Z_k) q, 0): only the sum C is kept.
// Without draft probabilities each draft is a point mass: R_k is p without the tokens
// refused here, Z_k = 1 - their probabilities, and x is accepted when u Z_k < R_k(x).
//
// The draw: the first x, in vocabulary order, with R(0) + ... + R(x) > u_sample * Z.
//
// Decisions lie next to borders, so sums are kept to about 1e-13 of the mass: the
// inputs are fp32 or bf16 (u q(x) and the widened values are exact in fp64), the walk's
// scalars are fp64, and a row is summed by each lane in pairs of fp32 (a value and what
// its rounding lost; every difference p - C q and every addition keeps its error term),
// joined in fp64.  The fp64 pipe does two operations per cycle and SM here: a row of
// fp64 additions took 286 us for 64 sequences of 129280 entries, where reading takes 10.
//
// Bound by memory: of T rows only those at which a draft is refused are read, p and q
// once each, and once more the sixteenth of a slice that holds the drawn token.  A
// cluster of CTAs shares a sequence (each a contiguous slice of the vocabulary), since
// one CTA alone reads ~0.1 TB/s; masses are exchanged through distributed shared
// memory.  Every CTA walks the tree alike (one warp, from shared memory).
#include <math.h>

#include "mla_internal.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTile = 256;          // vocabulary entries a warp reads at once, 8 per lane
constexpr int kFilterBits = 8192;   // one bit per group of 8 entries (modulo): may hold a refused token

struct VerifyArgs {
  const void *target, *draft;       // draft null: point masses
  int64_t row_stride;               // elements between rows
  const int32_t *tokens, *parents, *node_lens;
  const float *u_accept, *u_sample;
  int32_t *accept_len, *accept_idx, *out_tokens;
  int T, V;
  int* status;
  int cluster;                      // CTAs per sequence
};

// A probability as it counts: a negative value, an infinity or a NaN is no mass.
__device__ __forceinline__ float clean(float p) { return p > 0.f && p < INFINITY ? p : 0.f; }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// Entries [x, x + 8) of a row (x a multiple of 8); those at or past V are 0.
__device__ __forceinline__ void load8(const float* row, int x, int V, float (&v)[8]) {
  if (x + 8 <= V) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row + x));
    const float4 b = __ldg(reinterpret_cast<const float4*>(row + x + 4));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x + e < V ? row[x + e] : 0.f;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int x, int V, float (&v)[8]) {
  if (x + 8 <= V) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + x));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x + e < V ? widen(row[x + e]) : 0.f;
  }
}

// What is left of p: p - C q, or p without the refused tokens.
struct Residual {
  double C;                  // > 0: subtract C q
  int num_refused;           // > 0: these tokens are out (point-mass drafts)
  const int* refused;
  const uint32_t* filter;
};

// An unevaluated sum of two fp32 values, hi the sum rounded.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_diff(float a, float b) {     // a - b, exactly
  const float d = a - b, t = d - a;
  return {d, (a - (d - t)) - (b + t)};
}
__device__ __forceinline__ void add_to(Pair& s, Pair v) {
  const float t = s.hi + v.hi, b = t - s.hi;
  s.lo += ((s.hi - (t - b)) + (v.hi - b)) + v.lo;
  s.hi = t;
}
__device__ __forceinline__ Pair shfl_xor(Pair v, int o) {
  return {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double value(Pair v) { return (double)v.hi + (double)v.lo; }

// Entries [x, x + 8) of what is left.
template <typename T>
__device__ __forceinline__ void residual8(const T* p_row, const T* q_row, const Residual& r, int x, int V,
                                          Pair (&out)[8]) {
  float p[8];
  load8(p_row, x, V, p);
  if (r.C > 0.0) {
    float q[8];
    load8(q_row, x, V, q);
    if (r.C == 1.0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = two_diff(clean(p[e]), clean(q[e]));
    } else {
      const float ch = (float)r.C, cl = (float)(r.C - (double)ch);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float qe = clean(q[e]), h = ch * qe, l = fmaf(cl, qe, fmaf(ch, qe, -h));
        const Pair d = two_diff(clean(p[e]), h);
        const float lo = d.lo - l, hi = d.hi + lo;
        out[e] = {hi, lo - (hi - d.hi)};
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!(out[e].hi > 0.f)) out[e] = {0.f, 0.f};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = {clean(p[e]), 0.f};
  }
  if (r.num_refused > 0) {
    const int bit = (x >> 3) & (kFilterBits - 1);
    if ((r.filter[bit >> 5] >> (bit & 31)) & 1u) {
      for (int k = 0; k < r.num_refused; ++k) {
        const int e = r.refused[k] - x;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e == j) out[j] = {0.f, 0.f};
      }
    }
  }
}

// Part k of n of the tiles [t0, t1): contiguous, in order.
__device__ __forceinline__ void part_of(int t0, int t1, int k, int n, int* first, int* last) {
  const long long len = t1 - t0;
  *first = t0 + (int)(len * k / n);
  *last = t0 + (int)(len * (k + 1) / n);
}

// The masses of the warps' parts of the tiles [t0, t1) into wsum[] (the whole CTA).
template <typename T>
__device__ void part_masses(const T* p_row, const T* q_row, const Residual& r, int V, int t0, int t1, Pair* wsum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int first, last;
  part_of(t0, t1, w, kVerifyWarps, &first, &last);
  Pair s{0.f, 0.f};
#pragma unroll 2
  for (int t = first; t < last; ++t) {
    Pair v[8];
    residual8(p_row, q_row, r, t * kTile + 8 * lane, V, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) add_to(s, v[e]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) add_to(s, shfl_xor(s, o));
  __syncthreads();   // wsum's last readers are done
  if (lane == 0) wsum[w] = s;
  __syncthreads();
}

// One warp, lane k holding the mass m of part k (0 past the last): the part that holds
// the entry at which the running sum, `run` at first, passes `goal`; the last part with
// mass if rounding leaves none (-1: no mass).  run becomes the sum before that part.
__device__ __forceinline__ int find_part(double m, double* run, double goal) {
  const int lane = threadIdx.x & 31;
  double incl = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const unsigned some = __ballot_sync(0xffffffffu, m > 0.0);
  const unsigned hit = __ballot_sync(0xffffffffu, m > 0.0 && *run + incl > goal);
  const int k = hit ? __ffs(hit) - 1 : 31 - __clz(some);
  if (k >= 0) *run += __shfl_sync(0xffffffffu, incl - m, k);
  return k;
}

// One warp: the first entry of the tiles [t0, t1) whose running sum, from `run` on,
// passes `goal`; their last entry of positive mass if rounding leaves none.
template <typename T>
__device__ int warp_find(const T* p_row, const T* q_row, const Residual& r, int V, int t0, int t1, double run,
                         double goal) {
  const int lane = threadIdx.x & 31;
  int last = -1;
  for (int t = t0; t < t1; ++t) {
    Pair v[8], s{0.f, 0.f};
    residual8(p_row, q_row, r, t * kTile + 8 * lane, V, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      add_to(s, v[e]);
      if (v[e].hi > 0.f) last = t * kTile + 8 * lane + e;
    }
    double before = run;
    const double mine = value(s);
    int src = find_part(mine, &before, goal);
    // the lane found passes the goal, or is the last one with mass of a tile that does not
    const double after = before + __shfl_sync(0xffffffffu, mine, src < 0 ? 0 : src);
    if (src >= 0 && after > goal) {
      // its eight entries, one per lane
      Pair e8{0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const Pair x{__shfl_sync(0xffffffffu, v[e].hi, src), __shfl_sync(0xffffffffu, v[e].lo, src)};
        if (lane == e) e8 = x;
      }
      return t * kTile + 8 * src + find_part(value(e8), &before, goal);
    }
    if (src >= 0) run = after;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
  return last;
}

// What the walking warp tells the others.
struct Walk {
  int cur, count, nref, want_mass;
  double C;
};

// What warp 0 decides about the draw: the CTA (-1: nothing is left) and its warp's part.
struct Draw {
  int cta, part;
  double run, goal;
};

// One cluster of CTAs per sequence.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(VerifyArgs a) {
  extern __shared__ int smem[];      // tokens, parents, p(x), q(x), u per node; the path; refused tokens
  __shared__ Pair wsum[kVerifyWarps];
  __shared__ double slice[2][kMaxCluster];   // the CTAs' masses, by turns
  __shared__ uint32_t filter[kFilterBits / 32];
  __shared__ Walk s_walk;
  __shared__ int s_next;
  __shared__ Draw s_draw;
  ptx::cluster_sync_all();   // the other CTAs run: their shared memory may be written
  pdl_wait();
  pdl_trigger();
  const int rank = (int)ptx::cluster_ctarank(), size = a.cluster;
  const int b = blockIdx.x / size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = a.T;
  int* tok = smem;
  int* par = smem + N;
  float* px = reinterpret_cast<float*>(smem + 2 * N);
  float* qx = reinterpret_cast<float*>(smem + 3 * N);
  float* ua = reinterpret_cast<float*>(smem + 4 * N);
  int* path = smem + 5 * N;
  int* refused = smem + 6 * N;
  int n = a.node_lens ? a.node_lens[b] : N;
  bool bad = n < 0 || n > N;
  if (bad) n = 0;
  const T* target = static_cast<const T*>(a.target) + (size_t)b * N * a.row_stride;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + (size_t)b * N * a.row_stride : nullptr;
  for (int t = tid; t < n; t += kVerifyThreads) {
    const int x = a.tokens[(size_t)b * N + t], pr = a.parents[(size_t)b * N + t];
    // A node that can be accepted hangs on an earlier one and holds a token of the vocabulary.
    const bool fine = t > 0 && pr >= 0 && pr < t && x >= 0 && x < a.V;
    bad |= t > 0 && !fine;
    tok[t] = x;
    par[t] = fine ? pr : -1;
    ua[t] = a.u_accept[(size_t)b * N + t];
    px[t] = fine ? clean(widen(target[(size_t)pr * a.row_stride + x])) : 0.f;
    qx[t] = fine && draft ? clean(widen(draft[(size_t)pr * a.row_stride + x])) : 1.f;
  }
  for (int k = tid; k < kFilterBits / 32; k += kVerifyThreads) filter[k] = 0;
  if (bad && rank == 0) atomicCAS(a.status, 0, MLA_ERR_DEVICE_CHECK);
  __syncthreads();

  int t0, t1, turn = 0;
  part_of(0, (a.V + kTile - 1) / kTile, rank, size, &t0, &t1);
  // The mass of what is left of a row: lane k of warp 0 gets the mass of CTA k's slice
  // (fp64 from here on is one warp's: an instruction takes its pipe for 16 cycles).
  auto mass = [&](const T* p_row, const T* q_row, const Residual& r) -> double {
    part_masses(p_row, q_row, r, a.V, t0, t1, wsum);
    if (warp == 0) {
      const double mine = warp_sum(lane < kVerifyWarps ? value(wsum[lane]) : 0.0);
      if (lane < size) {
        const uint32_t to = ptx::map_to_cta(ptx::smem_addr(&slice[turn][rank]), lane);
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(mine) : "memory");
      }
    }
    __syncwarp();
    ptx::cluster_sync_all();
    const double m = warp == 0 && lane < size ? slice[turn][lane] : 0.0;
    turn ^= 1;
    return m;
  };

  // The walk (warp 0), stopping where a refusal asks for the mass left.
  int cur = 0, at = 0, count = n > 0 ? 1 : 0, nref = 0;
  double C = 0.0, Z = 1.0;
  bool stale = false;     // Z has to be summed anew
  if (tid == 0 && n > 0) path[0] = 0;
  while (true) {
    if (warp == 0) {
      int want = 0;
      while (n > 0) {
        // the next child of cur, in index order
        int child = -1;
        for (int base = at + 1; base < n; base += 32) {
          const unsigned m = __ballot_sync(0xffffffffu, base + lane < n && par[base + lane] == cur);
          if (m) { child = base + __ffs(m) - 1; break; }
        }
        if (child < 0) break;
        if (stale) { want = 1; break; }
        at = child;
        const double u = (double)ua[child], p = (double)px[child], q = (double)qx[child];
        double left = p - C * q;
        if (!draft) {
          bool again = false;
          for (int base = 0; base < nref; base += 32)
            again |= __any_sync(0xffffffffu, base + lane < nref && refused[base + lane] == tok[child]);
          left = again ? 0.0 : p;
        }
        if (left > 0.0 && u * q * Z < left) {
          cur = child;
          if (lane == 0) path[count] = child;
          ++count;
          C = 0.0; Z = 1.0; nref = 0;
        } else if (draft) {
          C += Z;
          stale = true;
        } else {
          if (left > 0.0) Z -= left;
          if (lane == 0) refused[nref] = tok[child];
          ++nref;
          __syncwarp();
        }
      }
      if (lane == 0) s_walk = Walk{cur, count, nref, want, C};
    }
    __syncthreads();
    const Walk w = s_walk;
    if (!w.want_mass) break;
    const Residual r{w.C, 0, nullptr, filter};
    const double m = mass(target + (size_t)w.cur * a.row_stride, draft + (size_t)w.cur * a.row_stride, r);
    if (warp == 0) {
      Z = warp_sum(m);
      stale = false;
    }
  }

  const Walk w = s_walk;
  int next = -1, writer = 0;
  if (n > 0) {
    for (int k = tid; k < w.nref; k += kVerifyThreads) {
      const int bit = (refused[k] >> 3) & (kFilterBits - 1);
      atomicOr(&filter[bit >> 5], 1u << (bit & 31));
    }
    __syncthreads();
    const T* p_row = target + (size_t)w.cur * a.row_stride;
    const T* q_row = draft ? draft + (size_t)w.cur * a.row_stride : nullptr;
    Residual r{w.C, w.nref, refused, filter};
    // Warp 0 decides: the CTA whose slice holds the drawn token, and the part of it.
    auto decide = [&](double m) {
      if (warp == 0) {
        const double total = warp_sum(m);
        Draw d{-1, -1, 0.0, (double)a.u_sample[b] * total};
        if (total > 0.0) {
          d.cta = find_part(m, &d.run, d.goal);
          if (d.cta == rank) d.part = find_part(lane < kVerifyWarps ? value(wsum[lane]) : 0.0, &d.run, d.goal);
        }
        if (lane == 0) s_draw = d;
      }
      __syncthreads();
    };
    decide(mass(p_row, q_row, r));
    if (s_draw.cta < 0 && (r.C > 0.0 || r.num_refused > 0)) {
      // nothing is left (p lies under the drafts everywhere): the draw is from p itself
      r.C = 0.0;
      r.num_refused = 0;
      const double m = mass(p_row, q_row, r);
      decide(m);
    }
    if (s_draw.cta >= 0) writer = s_draw.cta;
    if (s_draw.cta == rank) {
      part_of(t0, t1, s_draw.part, kVerifyWarps, &t0, &t1);
      part_masses(p_row, q_row, r, a.V, t0, t1, wsum);       // that part shared out again, and the token in it
      if (warp == 0) {
        double run = s_draw.run;
        const double goal = s_draw.goal;
        const int k = find_part(lane < kVerifyWarps ? value(wsum[lane]) : 0.0, &run, goal);
        part_of(t0, t1, k, kVerifyWarps, &t0, &t1);
        const int x = warp_find(p_row, q_row, r, a.V, t0, t1, run, goal);
        if (lane == 0) s_next = x;
      }
      __syncthreads();
      next = s_next;
    }
  }
  if (rank != writer) return;
  for (int t = tid; t < N; t += kVerifyThreads) {
    a.accept_idx[(size_t)b * N + t] = t < w.count ? path[t] : -1;
    a.out_tokens[(size_t)b * N + t] = t + 1 < w.count ? tok[path[t + 1]] : (t + 1 == w.count ? next : -1);
  }
  if (tid == 0) a.accept_len[b] = w.count;
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyCall& c, cudaStream_t st) {
  VerifyArgs a{c.target, c.draft, c.row_stride, c.tokens, c.parents, c.node_lens, c.u_accept, c.u_sample,
               c.accept_len, c.accept_idx, c.out_tokens, c.T, c.V, bmm_status_ptr(), 1};
  if (!a.status) return cudaErrorInvalidValue;
  // As many CTAs per sequence as stay resident at once (two per SM).
  const int slots = 2 * mla_device_sm_count();
  while (a.cluster < kMaxCluster && (long long)c.B * a.cluster * 2 <= slots) a.cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(c.B * a.cluster));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.dynamicSmemBytes = (size_t)c.T * 7 * sizeof(int);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return c.bf16 ? cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, a)
                : cudaLaunchKernelEx(&cfg, verify_kernel<float>, a);
}

}  // namespace mla
