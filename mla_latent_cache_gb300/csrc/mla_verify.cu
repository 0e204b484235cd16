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
// Decisions lie next to borders, so every sum, product and comparison is done in pairs of
// fp32 (a value and what its rounding lost, Dekker's and Knuth's error-free sums and
// products): sums are good to about 1e-13 of the mass, and u q(x) is exact.  fp64 itself
// is too slow here, at two operations per cycle and SM: 64 sequences of 129280 entries took
// 286 us with rows summed in fp64, where reading them takes 10.
//
// Bound by memory: of T rows only those at which a draft is refused are read, p and q
// once each, and once more the sixteenth of a slice that holds the drawn token.  A
// cluster of CTAs shares a sequence (each a contiguous slice of the vocabulary), since
// one CTA alone reads ~0.1 TB/s; masses are exchanged through distributed shared
// memory.  Every CTA walks the tree alike (one warp, from shared memory).  64 chains of 6
// over 129280 entries in fp32, p and q: 23.3 us, of which ~10 at the copy rate and the rest
// latency (nodes and their p, q 1.1, walk, exchange 1.8, search 3.8); 48 trees of 24 over
// 50257, point masses: 12.1 us; one chain of 5 over 32000 in bf16: 6.7 us.
#include <math.h>

#include <atomic>

#include "mla_internal.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTile = 256;          // vocabulary entries a warp reads at once, 8 per lane
constexpr int kFirst = 1 << 16;     // next to a parent's number (below kMaxTreeNodes)
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
    const float4 a = *reinterpret_cast<const float4*>(row + x);
    const float4 b = *reinterpret_cast<const float4*>(row + x + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x + e < V ? row[x + e] : 0.f;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int x, int V, float (&v)[8]) {
  if (x + 8 <= V) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + x);
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

// An unevaluated sum of two fp32 values, hi the sum rounded.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {      // a + b, exactly
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair quick_sum(float a, float b) {    // the same for |a| >= |b|
  const float s = a + b;
  return {s, b - (s - a)};
}
__device__ __forceinline__ Pair two_prod(float a, float b) {     // a b, exactly
  const float p = a * b;
  return {p, fmaf(a, b, -p)};
}
__device__ __forceinline__ void add_to(Pair& s, Pair v) {        // lo not carried into hi
  const Pair t = two_sum(s.hi, v.hi);
  s.lo += t.lo + v.lo;
  s.hi = t.hi;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair s = two_sum(a.hi, b.hi);
  const Pair t = two_sum(a.lo, b.lo);
  s = quick_sum(s.hi, s.lo + t.hi);
  return quick_sum(s.hi, s.lo + t.lo);
}
__device__ __forceinline__ Pair sub(Pair a, Pair b) { return add(a, {-b.hi, -b.lo}); }
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const Pair p = two_prod(a.hi, b.hi);
  return quick_sum(p.hi, p.lo + fmaf(a.hi, b.lo, a.lo * b.hi));
}
__device__ __forceinline__ Pair scaled(Pair a, float power_of_2) { return {a.hi * power_of_2, a.lo * power_of_2}; }
__device__ __forceinline__ bool less(Pair a, Pair b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }

// Masses, and what is compared with them, are held times 2^64: products with a number
// u >= 2^-24 and their error terms then stay in fp32's range for masses down to its least.
constexpr float kScale = 18446744073709551616.f, kUnscale = 1.f / kScale;
constexpr float kHalf = 4294967296.f;   // sqrt(kScale): shared by the factors of a product

// What is left of p: p - C q, or p without the refused tokens.
struct Residual {
  Pair C;                    // > 0: subtract C q
  int num_refused;           // > 0: these tokens are out (point-mass drafts)
  const int* refused;
  int cur;                   // the node after which p stands
};
// A CTA's shared state.  What is left stands here and not in an argument: a stack frame of
// a few words per thread is megabytes of local memory a launch (104 bytes: 27 -> 32 us for
// 64 sequences of 129280 entries).
struct Shared {
  Residual left;
  int want_mass, count;               // told by the walk
  int cta, t0, t1;                    // told by warp 0 about the draw: the CTA (-1: nothing is left), the tiles that hold the token
  Pair run, goal;                     // the mass before those tiles, and the one to pass
  int next;
  unsigned some_warps;                // bits of the warps that have mass
  unsigned some[kVerifyWarps];        // of a warp's lanes that have
  Pair wsum[kVerifyWarps];            // running sums over the CTA's warps
  Pair lsum[kVerifyThreads];          // running sums over a warp's lanes
  float2 slice[2][kMaxCluster];       // the CTAs' masses, by turns
  uint32_t filter[kFilterBits / 32];
};
__shared__ Shared sh;

// What is left of entries [x, x + 8), from p and (kQ: C > 0) q there.
template <bool kQ>
__device__ __forceinline__ void residual8(const float (&p)[8], const float (&q)[8], const Residual& r, int x,
                                          Pair (&out)[8]) {
  if (kQ) {
    if (r.C.hi == 1.f && r.C.lo == 0.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = quick_sum(clean(p[e]), -clean(q[e]));   // (p < q is cut to 0 below)
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float qe = clean(q[e]);
        const Pair cq = two_prod(r.C.hi, qe), d = two_sum(clean(p[e]), -cq.hi);
        out[e] = quick_sum(d.hi, d.lo - fmaf(r.C.lo, qe, cq.lo));
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
    if ((sh.filter[bit >> 5] >> (bit & 31)) & 1u) {
      for (int k = 0; k < r.num_refused; ++k) {
        const int e = r.refused[k] - x;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e == j) out[j] = {0.f, 0.f};
      }
    }
  }
}

// This lane's sum of what is left of the tiles [first, last).  One tile at a time: the kernel
// runs once through most of its code, so that what a longer body gains in loads in flight
// it loses in instructions to fetch (two tiles at once: 64 chains 23.2 -> 24.4 us, one chain
// 6.7 -> 8.2 us).
template <bool kQ, typename T>
__device__ __forceinline__ Pair sum_tiles(const T* p_row, const T* q_row, const Residual& r, int V, int first, int last) {
  Pair s{0.f, 0.f};
#pragma unroll 1
  for (int t = first; t < last; ++t) {
    const int x = t * kTile + 8 * (threadIdx.x & 31);
    float p[8], q[8];
    Pair v[8];
    load8(p_row, x, V, p);
    if (kQ) load8(q_row, x, V, q);
    residual8<kQ>(p, q, r, x, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) add_to(s, v[e]);
  }
  return s;
}

// Part k of n of the tiles [t0, t1): contiguous, in order.
__device__ __forceinline__ void part_of(int t0, int t1, int k, int n, int* first, int* last) {
  const long long len = t1 - t0;
  *first = t0 + (int)(len * k / n);
  *last = t0 + (int)(len * (k + 1) / n);
}

__device__ __forceinline__ Pair shfl(Pair v, int lane) {
  return {__shfl_sync(0xffffffffu, v.hi, lane), __shfl_sync(0xffffffffu, v.lo, lane)};
}
__device__ __forceinline__ Pair keep_if(bool keep, Pair v) { return {keep ? v.hi : 0.f, keep ? v.lo : 0.f}; }
// The running sums of the first `width` lanes' values (a power of two; later lanes hold no
// sum), ~110 cycles a step.  Every mass is summed so once, and the search for the drawn
// token takes what the sums left behind.
// (Called behind a branch that some lanes take, a warp goes through the steps in two parts
// that meet at every shuffle: 3300 cycles in place of 550, measured.  So what callers pass
// is chosen by selects, zeros are added where a lane has nothing to add, and one lane's
// stores are followed by __syncwarp.)
__device__ __noinline__ Pair warp_scan(Pair v, int width) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int o = 1; o < width; o <<= 1) {
    const Pair y{__shfl_up_sync(0xffffffffu, v.hi, o), __shfl_up_sync(0xffffffffu, v.lo, o)};
    v = add(v, keep_if(lane >= o, y));
  }
  return v;
}

// What is left of entry x alone (x < V).
template <typename T>
__device__ __forceinline__ Pair residual1(const T* p_row, const T* q_row, const Residual& r, int x) {
  Pair v{clean(widen(p_row[x])), 0.f};
  if (r.C.hi > 0.f) {
    const Pair cq = mul(r.C, {clean(widen(q_row[x])), 0.f});
    v = sub(v, cq);
    if (!(v.hi > 0.f)) v = {0.f, 0.f};
  }
  for (int k = 0; k < r.num_refused; ++k)
    if (r.refused[k] == x) v = {0.f, 0.f};
  return v;
}

// The masses (scaled) of what sh.left leaves of the tiles [t0, t1): the running sums over a
// warp's lanes into lsum[], which lanes have mass into some[], and (in warp 0, which alone
// reads them) the running sums over the warps' parts into wsum[].  The whole CTA.
template <typename T>
__device__ __noinline__ Pair part_masses(const T* p_row, const T* q_row, int V, int t0, int t1) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const Residual r = sh.left;
  int first, last;
  part_of(t0, t1, w, kVerifyWarps, &first, &last);
  Pair s = r.C.hi > 0.f ? sum_tiles<true>(p_row, q_row, r, V, first, last)
                        : sum_tiles<false>(p_row, q_row, r, V, first, last);
  s = scaled(quick_sum(s.hi, s.lo), kScale);
  const unsigned with_mass = __ballot_sync(0xffffffffu, s.hi > 0.f);
  s = warp_scan(s, 32);
  __syncthreads();   // the last readers of these arrays are done
  sh.lsum[threadIdx.x] = s;
  if (lane == 31) sh.wsum[w] = s;
  if (lane == 0) sh.some[w] = with_mass;
  __syncthreads();
  if (w == 0) {
    s = keep_if(lane < kVerifyWarps, sh.wsum[lane % kVerifyWarps]);
    const unsigned warps = __ballot_sync(0xffffffffu, s.hi > 0.f);
    s = warp_scan(s, kVerifyWarps);
    if (lane < kVerifyWarps) sh.wsum[lane] = s;
    if (lane == 0) sh.some_warps = warps;
    __syncwarp();
    s = shfl(s, kVerifyWarps - 1);
  }
  return s;      // warp 0: the CTA's mass
}

// One warp, lane k holding the running sum `incl` of the parts up to part k, those in the
// bits `some` with mass: the part that holds the entry at which the sum, `run` before these
// parts, passes `goal`; the last part with mass if rounding leaves none (-1: no mass).  And
// the sum before that part.
struct Found {
  int part;
  Pair run;
};
__device__ __noinline__ Found find_part(Pair incl, unsigned some, Pair run, Pair goal) {
  incl = add(run, incl);
  const unsigned hit = __ballot_sync(0xffffffffu, less(goal, incl)) & some;
  const int k = hit ? __ffs(hit) - 1 : 31 - __clz(some);
  const Pair before = shfl(incl, k > 0 ? k - 1 : 0);
  return {k, k > 0 ? before : run};
}

// One cluster of CTAs per sequence.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(VerifyArgs a) {
  extern __shared__ int smem[];      // tokens, parents, p(x), q(x), u per node; the path; refused tokens
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ptx::cluster_sync_all();   // the other CTAs run: their shared memory may be written
  pdl_wait();
  pdl_trigger();
  const int rank = (int)ptx::cluster_ctarank(), size = a.cluster;
  const int b = blockIdx.x / size;
  const int N = a.T;
  int* tok = smem;
  int* par = smem + N;               // | kFirst: accepted if it is its parent's first child tried
  float* px = reinterpret_cast<float*>(smem + 2 * N);
  float* qx = reinterpret_cast<float*>(smem + 3 * N);
  float* ua = reinterpret_cast<float*>(smem + 4 * N);
  int* path = smem + 5 * N;
  int* refused = smem + 6 * N;
  // (a thread's first node is asked for together with the count)
  int x_first = 0, pr_first = -1;
  if (tid < N) {
    x_first = a.tokens[(size_t)b * N + tid];
    pr_first = a.parents[(size_t)b * N + tid];
  }
  int n = a.node_lens ? a.node_lens[b] : N;
  const float us = a.u_sample[b];
  bool bad = n < 0 || n > N;
  if (bad) n = 0;
  const T* target = static_cast<const T*>(a.target) + (size_t)b * N * a.row_stride;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + (size_t)b * N * a.row_stride : nullptr;
  for (int t = tid; t < n; t += kVerifyThreads) {
    const int x = t == tid ? x_first : a.tokens[(size_t)b * N + t];
    const int pr = t == tid ? pr_first : a.parents[(size_t)b * N + t];
    // A node that can be accepted hangs on an earlier one and holds a token of the vocabulary.
    const bool fine = t > 0 && pr >= 0 && pr < t && x >= 0 && x < a.V;
    bad |= t > 0 && !fine;
    tok[t] = x;
    const float u = a.u_accept[(size_t)b * N + t];
    const float p = fine ? clean(widen(target[(size_t)pr * a.row_stride + x])) : 0.f;
    const float q = fine && draft ? clean(widen(draft[(size_t)pr * a.row_stride + x])) : 1.f;
    ua[t] = u;
    px[t] = p;
    qx[t] = q;
    const bool first = p > 0.f && less(scaled(two_prod(u * kHalf, q), kHalf), {p * kScale, 0.f});
    par[t] = fine ? pr | (first ? kFirst : 0) : -1;
  }
  for (int k = tid; k < kFilterBits / 32; k += kVerifyThreads) sh.filter[k] = 0;
  if (bad && rank == 0) atomicCAS(a.status, 0, MLA_ERR_DEVICE_CHECK);
  __syncthreads();

  int turn = 0;

  // The walk (warp 0), stopping where a refusal asks for the mass left; at its end the draw.
  int cur = 0, at = 0, count = 1, nref = 0;
  const Pair none{0.f, 0.f}, one{kScale, 0.f};
  Pair C = none, Z = one;   // Z scaled
  bool stale = false;       // Z has to be summed anew
  bool bare = false;        // the draw is from p itself
  if (tid == 0) path[0] = 0;
  while (n > 0) {
    if (warp == 0) {
      int want = 0;
      while (!bare) {
        // the next child of cur, in index order
        int child = -1;
        bool first = false;
        for (int base = at + 1; base < n; base += 32) {
          const int v = base + lane < n ? par[base + lane] : -1;
          const unsigned m = __ballot_sync(0xffffffffu, (v | kFirst) == (cur | kFirst));
          const unsigned f = __ballot_sync(0xffffffffu, v >= kFirst);
          if (m) {
            child = base + __ffs(m) - 1;
            first = (f >> (__ffs(m) - 1)) & 1u;
            break;
          }
        }
        if (child < 0) break;
        if (stale) { want = 1; break; }
        at = child;
        Pair left{px[child], 0.f};
        bool accepted = first;
        if (C.hi > 0.f || nref > 0) {        // others were refused here
          const float u = ua[child], q = qx[child];
          if (draft) {
            left = sub(left, mul(C, {q, 0.f}));
          } else {
            bool again = false;
            for (int base = 0; base < nref; base += 32)
              again |= __any_sync(0xffffffffu, base + lane < nref && refused[base + lane] == tok[child]);
            if (again) left = none;
          }
          left = scaled(left, kScale);
          accepted = left.hi > 0.f && less(mul(two_prod(u * kHalf, q), scaled(Z, 1.f / kHalf)), left);
        } else {
          left = scaled(left, kScale);
        }
        if (accepted) {
          cur = child;
          if (lane == 0) path[count] = child;
          __syncwarp();
          ++count;
          C = none; Z = one; nref = 0;
        } else if (draft) {
          C = add(C, scaled(Z, kUnscale));
          stale = true;
        } else {
          if (left.hi > 0.f) Z = sub(Z, left);
          if (lane == 0) refused[nref] = tok[child];
          ++nref;
          __syncwarp();
        }
      }
      for (int k = lane; k < nref; k += 32) {     // (at the walk's end only: nobody looks before)
        const int bit = (refused[k] >> 3) & (kFilterBits - 1);
        if (!want && !bare) atomicOr(&sh.filter[bit >> 5], 1u << (bit & 31));
      }
      __syncwarp();
      if (lane == 0) {
        sh.left = Residual{bare ? none : C, bare || want ? 0 : nref, refused, cur};
        sh.want_mass = want;
        sh.count = count;
      }
    }
    __syncthreads();
    const bool want_mass = sh.want_mass;
    // The mass (scaled) of what is left of the row: lane k of warp 0 gets that of CTA k's slice.
    int t0, t1;
    part_of(0, (a.V + kTile - 1) / kTile, rank, size, &t0, &t1);
    const Pair mine = part_masses(target + (size_t)sh.left.cur * a.row_stride,
                                  draft ? draft + (size_t)sh.left.cur * a.row_stride : nullptr, a.V, t0, t1);
    if (warp == 0 && lane < size) {
      const uint32_t to = ptx::map_to_cta(ptx::smem_addr(&sh.slice[turn][rank]), lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(mine.hi), "f"(mine.lo) : "memory");
    }
    __syncwarp();
    ptx::cluster_sync_all();
    if (warp == 0) {
      const float2 s = sh.slice[turn][lane % kMaxCluster];
      const Pair m = keep_if(lane < size, {s.x, s.y});
      const unsigned some = __ballot_sync(0xffffffffu, m.hi > 0.f);
      const Pair slices = warp_scan(m, kMaxCluster);
      Z = shfl(slices, kMaxCluster - 1);
      stale = false;
      // the draw: the CTA whose slice holds the token, if this was the walk's end
      if (!want_mass) {
        const Pair goal = mul(Z, {us, 0.f});
        const Found f = find_part(slices, some, none, goal);
        if (lane == 0) {
          sh.cta = f.part;
          sh.t0 = t0;
          sh.t1 = t1;
          sh.run = f.run;
          sh.goal = goal;
        }
      }
    }
    turn ^= 1;
    __syncthreads();
    if (want_mass) continue;
    if (sh.cta >= 0 || bare) break;
    bare = true;          // nothing is left: p lies under the drafts everywhere
  }

  int next = -1, writer = 0;
  const int count_all = n > 0 ? sh.count : 0;
  if (n > 0) {
    if (sh.cta >= 0) writer = sh.cta;
    if (sh.cta == rank) {
      // The part of the tiles that holds the token, shared out again until each warp has one
      // tile at most; then its warp's lane, and that lane's entry.
      const T* p_row = target + (size_t)sh.left.cur * a.row_stride;
      const T* q_row = draft ? draft + (size_t)sh.left.cur * a.row_stride : nullptr;
      while (true) {
        const int first = sh.t0, last = sh.t1;
        __syncthreads();
        if (warp == 0) {
          const Pair goal = sh.goal;
          const Found w = find_part(sh.wsum[lane % kVerifyWarps], sh.some_warps, sh.run, goal);
          const int k = max(0, w.part);
          int f, l;
          part_of(first, last, k, kVerifyWarps, &f, &l);
          if (last - first <= kVerifyWarps) {
            const Found in_tile = find_part(sh.lsum[32 * k + lane], sh.some[k], w.run, goal);
            const int x = f * kTile + 8 * max(0, in_tile.part);
            // (a lane past the tile's eight, or the vocabulary, looks at the last entry for nothing)
            const int mine = min(x + min(lane, 7), a.V - 1);
            const Pair e = keep_if(mine == x + lane, scaled(residual1(p_row, q_row, sh.left, mine), kScale));
            const unsigned some = __ballot_sync(0xffffffffu, e.hi > 0.f);
            const Found entry = find_part(warp_scan(e, 8), some, in_tile.run, goal);
            if (lane == 0) sh.next = x + max(0, entry.part);
          }
          if (lane == 0) {
            sh.t0 = f;
            sh.t1 = l;
            sh.run = w.run;
          }
        }
        __syncthreads();
        if (last - first <= kVerifyWarps) break;
        part_masses(p_row, q_row, a.V, sh.t0, sh.t1);
      }
      next = sh.next;
    }
  }
  if (rank != writer) return;
  for (int t = tid; t < N; t += kVerifyThreads) {
    a.accept_idx[(size_t)b * N + t] = t < count_all ? path[t] : -1;
    a.out_tokens[(size_t)b * N + t] = t + 1 < count_all ? tok[path[t + 1]] : (t + 1 == count_all ? next : -1);
  }
  if (tid == 0) a.accept_len[b] = count_all;
}

void cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&attr)[2], int clusters, int size, size_t smem,
                    cudaStream_t st) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3((unsigned)(clusters * size));
  cfg->blockDim = dim3(kVerifyThreads);
  cfg->dynamicSmemBytes = smem;
  cfg->stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// CTAs per sequence: as many as leave all B clusters resident at once (a cluster lies within
// a group of SMs, so that is not the slots by the size: 48 clusters of 6 take 16.0 us where
// 48 of 4 take 12.3, and 44 of 6 take 16.8 where 44 of 4 take 19.4).
int cluster_size(int B) {
  // Filled on first use per device; concurrent first calls compute and store the same values.
  static std::atomic<int> resident[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  for (int size = kMaxCluster; size > 1; --size) {
    int n = resident[dev][size].load(std::memory_order_relaxed);
    if (n == 0) {
      cudaLaunchConfig_t cfg;
      cudaLaunchAttribute attr[2];
      cluster_config(&cfg, attr, 64, size, kMaxTreeNodes * 7 * sizeof(int), nullptr);
      if (cudaOccupancyMaxActiveClusters(&n, verify_kernel<float>, &cfg) != cudaSuccess || n <= 0) n = -1;
      resident[dev][size].store(n, std::memory_order_relaxed);
    }
    if (n >= B) return size;
  }
  return 1;
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyCall& c, cudaStream_t st) {
  VerifyArgs a{c.target, c.draft, c.row_stride, c.tokens, c.parents, c.node_lens, c.u_accept, c.u_sample,
               c.accept_len, c.accept_idx, c.out_tokens, c.T, c.V, bmm_status_ptr(), cluster_size(c.B)};
  if (!a.status) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  cluster_config(&cfg, attr, c.B, a.cluster, (size_t)c.T * 7 * sizeof(int), st);
  return c.bf16 ? cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, a)
                : cudaLaunchKernelEx(&cfg, verify_kernel<float>, a);
}

}  // namespace mla
