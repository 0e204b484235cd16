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
// Decisions lie next to borders, so every product and sum is fp64 (the inputs are fp32
// or bf16, so u q(x) and the widened values are exact).
#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kVerifyThreads = 1024;
constexpr int kVerifyWarps = kVerifyThreads / 32;
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
};

// A probability as it counts: a negative value or a NaN is no mass.
__device__ __forceinline__ float clean(float p) { return p > 0.f ? p : 0.f; }
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

template <typename T>
__device__ __forceinline__ void residual8(const T* p_row, const T* q_row, const Residual& r, int x, int V,
                                          double (&out)[8]) {
  float p[8];
  load8(p_row, x, V, p);
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = (double)clean(p[e]);
  if (r.C > 0.0) {
    float q[8];
    load8(q_row, x, V, q);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double d = out[e] - r.C * (double)clean(q[e]);
      out[e] = d > 0.0 ? d : 0.0;
    }
  }
  if (r.num_refused > 0) {
    const int bit = (x >> 3) & (kFilterBits - 1);
    if ((r.filter[bit >> 5] >> (bit & 31)) & 1u) {
      for (int k = 0; k < r.num_refused; ++k) {
        const int e = r.refused[k] - x;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e == j) out[j] = 0.0;
      }
    }
  }
}

// Tiles [first, last) of warp w: the row is cut into contiguous runs of tiles.
__device__ __forceinline__ void warp_tiles(int V, int w, int* first, int* last) {
  const int n = (V + kTile - 1) / kTile;
  *first = (int)((long long)n * w / kVerifyWarps);
  *last = (int)((long long)n * (w + 1) / kVerifyWarps);
}

// The mass of each warp's run into wsum[], and the whole mass (every thread).
template <typename T>
__device__ double block_mass(const T* p_row, const T* q_row, const Residual& r, int V, double* wsum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int t0, t1;
  warp_tiles(V, w, &t0, &t1);
  double s = 0.0;
  for (int t = t0; t < t1; ++t) {
    double v[8];
    residual8(p_row, q_row, r, t * kTile + 8 * lane, V, v);
    s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();   // wsum's last readers are done
  if (lane == 0) wsum[w] = s;
  __syncthreads();
  double total = 0.0;
  for (int k = 0; k < kVerifyWarps; ++k) total += wsum[k];
  return total;
}

// One warp: the first entry of its run whose running sum, from `run` on, passes `goal`;
// the run's last entry of positive mass if rounding leaves none (-1 if it has no mass).
template <typename T>
__device__ int warp_find(const T* p_row, const T* q_row, const Residual& r, int V, int w, double run, double goal) {
  const int lane = threadIdx.x & 31;
  int t0, t1, last = -1;
  warp_tiles(V, w, &t0, &t1);
  for (int t = t0; t < t1; ++t) {
    const int x = t * kTile + 8 * lane;
    double v[8];
    residual8(p_row, q_row, r, x, V, v);
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s += v[e];
      if (v[e] > 0.0) last = x + e;
    }
    double incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, run + incl > goal && s > 0.0);
    if (hit) {
      const int src = __ffs(hit) - 1;
      int found = -1;
      double acc = run + (incl - s);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc += v[e];
        if (v[e] > 0.0 && (found < 0 || !(found & 0x40000000))) {
          // the first entry that passes the goal is final (marked); until then the last positive one stands
          found = (x + e) | (acc > goal ? 0x40000000 : 0);
        }
      }
      return __shfl_sync(0xffffffffu, found, src) & 0x3FFFFFFF;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
  return last;
}

// One CTA per sequence.  Every warp walks the tree alike, from shared memory; the whole
// CTA sums a row whenever the walk asks for the mass left after a refusal.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(VerifyArgs a) {
  extern __shared__ int smem[];      // tokens, parents, p(x), q(x) per node; the path; refused tokens
  __shared__ double wsum[kVerifyWarps];
  __shared__ uint32_t filter[kFilterBits / 32];
  __shared__ int s_next;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int N = a.T;
  int* tok = smem;
  int* par = smem + N;
  float* px = reinterpret_cast<float*>(smem + 2 * N);
  float* qx = reinterpret_cast<float*>(smem + 3 * N);
  float* ua = reinterpret_cast<float*>(smem + 4 * N);
  int* path = smem + 5 * N;
  int* refused = smem + 6 * N;
  int n = a.node_lens ? a.node_lens[b] : N;
  const bool bad_len = n < 0 || n > N;
  if (bad_len) n = 0;
  const T* target = static_cast<const T*>(a.target) + (size_t)b * N * a.row_stride;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + (size_t)b * N * a.row_stride : nullptr;
  bool bad = bad_len;
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
  if (bad) atomicCAS(a.status, 0, MLA_ERR_DEVICE_CHECK);
  __syncthreads();

  int cur = 0, at = 0, count = n > 0 ? 1 : 0, nref = 0;
  double C = 0.0, Z = 1.0;
  bool stale = false;     // Z has to be summed anew
  if (tid == 0 && n > 0) path[0] = 0;
  while (n > 0) {
    // the next child of cur, in index order
    int child = -1;
    for (int base = at + 1; base < n; base += 32) {
      const unsigned m = __ballot_sync(0xffffffffu, base + lane < n && par[base + lane] == cur);
      if (m) { child = base + __ffs(m) - 1; break; }
    }
    if (child < 0) break;
    at = child;
    const double u = (double)ua[child], p = (double)px[child], q = (double)qx[child];
    double left;
    if (draft) {
      if (stale) {
        const Residual r{C, 0, nullptr, filter};
        Z = block_mass(target + (size_t)cur * a.row_stride, draft + (size_t)cur * a.row_stride, r, a.V, wsum);
        stale = false;
      }
      left = p - C * q;
    } else {
      bool again = false;
      for (int base = 0; base < nref; base += 32)
        again |= __any_sync(0xffffffffu, base + lane < nref && refused[base + lane] == tok[child]);
      left = again ? 0.0 : p;
    }
    if (left > 0.0 && u * q * Z < left) {
      cur = child;
      if (tid == 0) path[count] = child;
      ++count;
      C = 0.0; Z = 1.0; nref = 0; stale = false;
    } else if (draft) {
      C += Z;
      stale = true;
    } else {
      if (left > 0.0) Z -= left;
      __syncthreads();     // the list's readers are done
      if (tid == 0) refused[nref] = tok[child];
      ++nref;
      __syncthreads();
    }
  }
  __syncthreads();

  int next = -1;
  if (n > 0) {
    for (int k = tid; k < nref; k += kVerifyThreads) {
      const int bit = (refused[k] >> 3) & (kFilterBits - 1);
      atomicOr(&filter[bit >> 5], 1u << (bit & 31));
    }
    __syncthreads();
    const T* p_row = target + (size_t)cur * a.row_stride;
    const T* q_row = draft ? draft + (size_t)cur * a.row_stride : nullptr;
    Residual r{C, nref, refused, filter};
    double total = block_mass(p_row, q_row, r, a.V, wsum);
    if (!(total > 0.0)) {
      // nothing is left (p lies under the drafts everywhere): the draw is from p itself
      r.C = 0.0;
      r.num_refused = 0;
      total = block_mass(p_row, q_row, r, a.V, wsum);
    }
    if (total > 0.0) {
      const double goal = (double)a.u_sample[b] * total;
      double run = 0.0;
      int w = -1, last = -1;
      double run_w = 0.0, run_last = 0.0;
      for (int k = 0; k < kVerifyWarps; ++k) {
        if (wsum[k] > 0.0) { last = k; run_last = run; }
        if (w < 0 && wsum[k] > 0.0 && run + wsum[k] > goal) { w = k; run_w = run; }
        run += wsum[k];
      }
      if (w < 0) { w = last; run_w = run_last; }
      if (warp == w) {
        const int x = warp_find(p_row, q_row, r, a.V, w, run_w, goal);
        if (lane == 0) s_next = x;
      }
      __syncthreads();
      next = s_next;
    }
  }
  for (int t = tid; t < N; t += kVerifyThreads) {
    a.accept_idx[(size_t)b * N + t] = t < count ? path[t] : -1;
    a.out_tokens[(size_t)b * N + t] = t + 1 < count ? tok[path[t + 1]] : (t + 1 == count ? next : -1);
  }
  if (tid == 0) a.accept_len[b] = count;
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyCall& c, cudaStream_t st) {
  VerifyArgs a{c.target, c.draft, c.row_stride, c.tokens, c.parents, c.node_lens, c.u_accept, c.u_sample,
               c.accept_len, c.accept_idx, c.out_tokens, c.T, c.V, bmm_status_ptr()};
  if (!a.status) return cudaErrorInvalidValue;
  const size_t smem = (size_t)c.T * 7 * sizeof(int);
  return c.bf16 ? launch_pdl(verify_kernel<__nv_bfloat16>, dim3(c.B), dim3(kVerifyThreads), smem, st, a)
                : launch_pdl(verify_kernel<float>, dim3(c.B), dim3(kVerifyThreads), smem, st, a);
}

}  // namespace mla
