// Sampling: the next token of each row of logits from a given random number, after
// temperature, min-p, top-k and top-p; and the probabilities that these leave.
//
// Rule, per row.  The tokens stand in order, the larger logit first and the lower index
// first among equals; e_i = exp((l_i - l_max) / temperature), so that the first has e = 1.
// Each filter keeps a leading part of what the one before left: min-p the tokens with
// e_i >= min_p; top-k the first k of those; top-p, with Z their sum, those before which the
// sum is less than top_p Z.  With M the sum of what is left, the token is the first whose
// running sum passes u M.  All three cuts are one search: the first token, in the order, at
// which the running sum of weights (1 for top-k, else the mass) reaches W.
//
// Masses are integers: e_i is taken in pairs of fp32 values (good to about 2^-45) and
// rounded to a multiple of 2^-44.  Sums of integers do not depend on their order, so that
// every sum, and with it every decision, is the same however the work is shared out, and
// comparisons with top_p Z and u M (128-bit products) are exact.  Decisions lie next to
// borders: fp32 sums (1e-7) would miss one in a hundred of a large vocabulary's.
//
// Nothing is sorted but a border's neighbourhood.  A cluster of CTAs takes a row, each a
// slice of it, and goes over it (from the L2 after the first time): for the maximum; for a
// histogram of masses (45-bit integers in three 15-bit limbs, whose 32-bit sums shared memory adds
// natively) over 2944 buckets of falling logits, 64 to a factor of 2; and for the tokens of the
// buckets that hold the borders, which one CTA puts in order.  A bucket of more than it can take is
// divided again, by key, until there is one key left, and equal keys are counted in index
// order.  Rows of which top-k or min-p leaves few go without the histogram of masses: their
// tokens' range follows from the settings and the threads' largest logits.
//
// What bounds it: 82 instructions a token of a row with a histogram of masses (issued on every cycle:
// 129280 tokens of 32 rows take 21 of 60 thousand cycles), and for every row 14 to 20
// thousand cycles of phases that wait for one another: the first loads, five barriers of the
// cluster, instructions that are fetched to be run once.  Measured: one bf16 row of 32000, top-k
// and top-p, 9.0 us; 64 fp32 rows of 129280 with mixed settings 41 us; 32 of them without filters 31 us; 96 rows
// of 50257 with top-p and their probabilities 50 us.  (A first form, which sorted nothing either but took
// double precision, one CTA a row and a pass per border: 611, 3015, 1823, 1230 us.)
#include <limits.h>
#include <math.h>
#include <stddef.h>

#include <atomic>

#include "mla_internal.cuh"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMassBits = 44;
constexpr int kTable = 1024;          // 2^(-j / 1024)
constexpr int kPerOctave = 64;        // buckets
constexpr int kOctaves = 46;
constexpr int kBuckets = kOctaves * kPerOctave;
// Buckets that can hold a mass: places are rounded to nearest, so that the first half place of bucket 45
// * 64 lies within 45 octaves, where a mass is just above 2^-45 and becomes one unit of 2^-44; the next
// bucket begins 15.5 places past them, at 0.495 units, which become none.
constexpr int kMassBuckets = (kMassBits + 1) * kPerOctave + 1;
constexpr float kFloorOctaves = 45.5f;   // what is further off has no mass (less than half of 2^-44)
constexpr int kList = 1024;           // tokens that one CTA sorts
constexpr int kGroup = 8;             // tokens a thread takes at once
constexpr int kFlush = 1 << 16;       // tokens after which a bucket's limbs are carried over
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a sum's low bits are the nearest integer

__device__ __forceinline__ void report(int* status) { atomicCAS(status, 0, MLA_ERR_DEVICE_CHECK); }

// Keys order logits: key(a) > key(b) where a > b, +0 and -0 alike; 0 for -inf and NaN (out).
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t x = __float_as_uint(l + 0.f);      // -0 becomes 0
  if (!(l > -INFINITY)) return 0u;
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// e = exp((l - max) / temperature) as a pair of fp32 values: 2^-t, t = (max - l) c, c =
// log2(e) / temperature as a pair.  t = j / 1024 + s with |s| <= 2^-11, 2^-s = 1 + z + z^2 / 2 +
// z^3 / 6 (z = -s ln 2, |z| < 2^-11.5: the next term is below 2^-50) and 2^(-j / 1024) from a
// table, its octaves taken off the exponents.  Off by 2^-45 at most, and by 2^-37 of itself.
//   The pass over a row's masses is bound by the fp32 pipes (an integer multiply-add, and a
// packed operation on two values, hold them for two cycles, measured), so that it counts
// how many operations this takes.
struct Scale {
  float max, ch, cl;
  // Logits below the floor (45.5 octaves off the maximum, or a little more) have no mass, and are
  // taken as it.  Rows for which fp32 has no such value, or a coarse one (temperatures of 10^35
  // or, by the maximum's last bit, of less than 23 of those), are taken token by token (wild).
  float floor;
  bool wild;
};
struct Term {
  float hi, lo;
  uint32_t place;            // kMagicBits + j
};
constexpr uint32_t kMagicBits = 0x4B400000u;        // of kMagic
__device__ __forceinline__ float octaves_off(float l, const Scale& sc) {
  // (as the pair below: the larger of max and -l first)
  return (fmaxf(sc.max, -l) + fminf(sc.max, -l)) * sc.ch;
}
__device__ __forceinline__ uint32_t place_of(float th) { return __float_as_uint(fmaf(th, (float)kTable, kMagic)); }
__device__ __forceinline__ int bucket_at(uint32_t place) { return (int)((place - kMagicBits) / (kTable / kPerOctave)); }
__device__ __forceinline__ int bucket_of(float l, const Scale& sc) {      // (NaN: the floor's)
  return bucket_at(place_of(fminf(octaves_off(fmaxf(l, sc.floor), sc), kFloorOctaves + 0.25f)));
}
// A range of logits that holds those of buckets [first, last], and few others: two comparisons a
// token, the bucket itself is worked out for what is in the range.  (Roundings of the
// octaves and of the quotient here: 2^-22 of them, the factors are wider.)
struct Range {
  float low, high;
  __device__ __forceinline__ bool has(float l) const { return l >= low && l <= high; }
};
__device__ __forceinline__ Range range_of(int first, int last, const Scale& sc) {
  constexpr int kStep = kTable / kPerOctave;
  const bool all = sc.wild || sc.ch > 1e30f;        // (beyond: quotients that are not normal)
  const float unit = (1.f / kTable) / sc.ch;
  const bool from_top = all || first <= 0, to_floor = all || last >= (int)kFloorOctaves * kPerOctave;
  return {to_floor ? -INFINITY : __fsub_rd(sc.max, (float)(kStep * (last + 1) + 1) * unit * (1.f + 0x1p-20f)),
          from_top ? INFINITY : __fsub_ru(sc.max, (float)(kStep * first - 1) * unit * (1.f - 0x1p-20f))};
}
// For logits of up to 60 octaves off.
__device__ __forceinline__ Term term_of(float l, const Scale& sc, const float2* table) {
  // max - l, exactly: whichever of max and -l is larger, as values, is so in magnitude (max >= l)
  const float x = fmaxf(sc.max, -l), y = fminf(sc.max, -l), d = x + y, dl = y - (d - x);
  const float th = d * sc.ch, tl = fmaf(d, sc.ch, -th) + fmaf(d, sc.cl, dl * sc.ch);
  const float jm = fmaf(th, (float)kTable, kMagic);
  const float s = fmaf(jm - kMagic, -1.f / kTable, th);   // exact
  constexpr float kLn2 = 0.693147182464599609375f, kLn2Low = -1.904654299957767e-9f;   // ln 2 = kLn2 + kLn2Low
  const float zh = s * -kLn2;
  const float zl = fmaf(s, -kLn2Low, fmaf(tl, -kLn2, fmaf(s, -kLn2, -zh)));
  const float rest = fmaf(zh, fmaf(zh, fmaf(zh, 1.f / 6.f, 0.5f), zl), zl);             // 2^-s = 1 + zh + rest
  // The place's bits past the tenth, shifted to an exponent's place, are the octaves (those of
  // kMagicBits fall out), and the table's entries have the other ten added there.
  const uint32_t place = __float_as_uint(jm), down = place << 13;
  const float2 tb = table[place & (kTable - 1)];
  const float Th = __uint_as_float(__float_as_uint(tb.x) - down), Tl = __uint_as_float(__float_as_uint(tb.y) - down);
  const float rh = fmaf(Th, zh, Th);
  return {rh, fmaf(Th, zh, Th - rh) + fmaf(Th, rest, fmaf(Tl, zh, Tl)), place};
}
// Whether min-p leaves the token out: by the pair, whose mass may be rounded past the bound.
__device__ __forceinline__ bool below(const Term& x, float min_p) { return (x.hi - min_p) + x.lo < 0.f; }
// The pair as a multiple of 2^-44, rounded to nearest.
__device__ __forceinline__ u64 fixed_of(float hi, float lo) {
  const float a = hi + 2.f;                         // units of 2^-22
  const float low = (hi - (a - 2.f)) + lo;          // |low| < 2^-22
  const uint32_t x = __float_as_uint(a) - __float_as_uint(2.f);
  // x 2^22 + (low 2^44, whose bits are kMagicBits and it)
  const u64 high = ((u64)(x >> 10) << 32) | (x << 22);
  return high + (__float_as_uint(fmaf(low, 17592186044416.f, kMagic)) - (u64)kMagicBits);
}
// The table, by products of its 32nd entries and its first 32, those by products of the roots.
// (The low parts are never 0, so that octaves can be taken off their exponents too.)
__device__ __forceinline__ float2 times(float2 a, float rh, float rl) {
  const float p = a.x * rh, e = fmaf(a.x, rh, -p) + fmaf(a.x, rl, a.y * rh), h = p + e;
  return make_float2(h, e - (h - p));
}
__device__ __forceinline__ float2 power_of_roots(int j) {        // 2^(-j / 1024)
  constexpr double kRoots[10] = {0.99932332750265075236, 0.99864711289097017358, 0.99729605608547012625, 0.99459942348363317565,
                                 0.98922801319397548413, 0.97857206208770013451, 0.95760328069857364694, 0.91700404320467123175,
                                 0.84089641525371454303, 0.70710678118654752440};       // 2^(-1/1024), 2^(-1/512) .. 2^(-1/2)
  float2 v = make_float2(1.f, 0.f);
#pragma unroll
  for (int k = 0; k < 10; ++k) {
    const float rh = (float)kRoots[k], rl = (float)(kRoots[k] - (double)rh);
    if ((j >> k) & 1) v = times(v, rh, rl);
  }
  return v;
}
__device__ __forceinline__ float2 table_entry(float2 v, int j) {
  if (v.y == 0.f) v.y = 0x1p-60f;
  return make_float2(__uint_as_float(__float_as_uint(v.x) + (j << 13)), __uint_as_float(__float_as_uint(v.y) + (j << 13)));
}

// floor(f 2^64) of a number f in [0, 1); 0 for others below
__device__ __forceinline__ u64 fraction(float f) {
  if (!(f > 0.f)) return 0;
  const uint32_t x = __float_as_uint(f);
  const int e = (int)(x >> 23);                     // f = m 2^(e - 150)
  const u64 m = (x & 0x7FFFFFu) | 0x800000u;
  return e >= 86 ? m << (e - 86) : e > 62 ? m >> (86 - e) : 0;
}
// The least integer not below f Z, and the least above f Z.
__device__ __forceinline__ u64 reach(float f, u64 Z) {
  const u64 x = fraction(f);
  const u64 w = __umul64hi(x, Z) + (x * Z != 0);
  return w < 1 ? 1 : w;
}
__device__ __forceinline__ u64 pass(float f, u64 Z) { return __umul64hi(fraction(f), Z) + 1; }

// a / b as a pair, of pairs
__device__ __forceinline__ float2 pair_divide(float ah, float al, float bh, float bl) {
  const float q = ah / bh;
  return make_float2(q, (fmaf(-q, bh, ah) + fmaf(-q, bl, al)) / bh);
}

// What the CTAs tell each other about a place in the order.
struct Found {
  u64 before, mass_before;   // weight and mass of the buckets before
  u64 mass;                  // of the bucket
  int bucket;
  unsigned count;            // of the bucket (where counts were taken)
};
struct Border {
  u64 mass;                  // up to the token, itself included
  uint32_t key;
  int index;
};
// The same place in another CTA's shared memory.
template <typename X>
__device__ __forceinline__ X* in_cta(X* p, int rank) {
  X* r;
  asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
  return r;
}

// Entries [8 g, 8 g + 8) of a row; those at or past V are out (-inf).
__device__ __forceinline__ void load8(const float* row, int g, int V, float (&v)[kGroup]) {
  const int x = kGroup * g;
  if (x + kGroup <= V) {
    const float4 a = *reinterpret_cast<const float4*>(row + x), b = *reinterpret_cast<const float4*>(row + x + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < kGroup; ++e) v[e] = x + e < V ? row[x + e] : -INFINITY;
  }
}
__device__ __forceinline__ float entry(const float* row, int x) { return row[x]; }
__device__ __forceinline__ float entry(const __nv_bfloat16* row, int x) { return __bfloat162float(row[x]); }
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int g, int V, float (&v)[kGroup]) {
  const int x = kGroup * g;
  if (x + kGroup <= V) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + x);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kGroup; ++e) v[e] = x + e < V ? entry(row, x + e) : -INFINITY;
  }
}

// A row as its CTA sees it.  It stands in shared memory, and functions copy what they use: a
// stack frame per thread would be megabytes of local memory a launch.
struct Row {
  const void* logits;
  int V, g0, g1;             // this CTA's groups of eight tokens: [g0, g1)
  int rank, size;
  bool trigger;              // the next kernel may come when the tokens are picked
  bool carried;              // the slices are of more than kFlush tokens (the same for all CTAs)
  bool infinite;             // the maximum is +inf: those tokens are equal, no others count
  Scale scale;
  float min_p;               // 0: off
  float cut;                 // the last token kept so far: logit and index
  int cut_index;

  __device__ __forceinline__ void barrier() const {
    if (size == 1) {
      __syncthreads();
    } else {
      __syncwarp();
      ptx::cluster_sync_all();
    }
  }
  __device__ __forceinline__ bool kept(float l, int i) const { return l > cut || (l == cut && i <= cut_index); }
  __device__ __forceinline__ float clean(float l) const { return infinite ? (l == INFINITY ? 0.f : -INFINITY) : l; }
  // f(eight logits, group) for the groups [first, last) of this CTA; the next ones are asked for
  // before f is called.
  template <typename T, typename F>
  __device__ __forceinline__ void each(int first, int last, F f) const {
    int g = first + threadIdx.x;
    if (g >= last) return;
    const T* from = static_cast<const T*>(logits);
    float next[kGroup];
    load8(from, g, V, next);
#pragma unroll 1
    do {
      float v[kGroup];
#pragma unroll
      for (int e = 0; e < kGroup; ++e) v[e] = next[e];
      if (infinite) {
#pragma unroll
        for (int e = 0; e < kGroup; ++e) v[e] = clean(v[e]);
      }
      const int at = g;
      g += kThreads;
      if (g < last) load8(from, g, V, next);
      f(v, at);
    } while (g < last);
  }
};

struct Sm {
  Row row;
  float2 table[kTable];
  alignas(16) unsigned count[kBuckets], limb[3][kBuckets];
  u64 carried[kBuckets];     // limbs carried over (slices of more than kFlush tokens)
  alignas(16) u64 pick[kList];           // this CTA's tokens of the border's buckets: key, ~index
  union {
    alignas(16) u64 list[kList];         // all CTAs' (the first CTA's), sorted
    float2 roots[64];        // (while the table is made)
  };
  u64 sum[kList];            // their running weights
  alignas(16) u64 omass[kMaxCluster][kOctaves];      // the CTAs' masses and counts, octave by octave
  alignas(16) unsigned ocount[kMaxCluster][kOctaves];
  alignas(16) u64 omass_run[kOctaves];   // their running sums
  alignas(16) unsigned ocount_run[kOctaves];
  alignas(16) u64 bmass[kMaxCluster][kPerOctave];     // the CTAs' buckets of an octave
  alignas(16) unsigned bcount[kMaxCluster][kPerOctave];
  u64 part[2 * kWarps];
  float fpart[kWarps], max[kMaxCluster];
  unsigned picked[kMaxCluster];
  int limit[kMaxCluster];
  Found found[2];
  Border border;
  unsigned n;                // picked here
  int at;
  uint32_t klo, khi;
};

static_assert(offsetof(Sm, pick) % 16 == 0 && offsetof(Sm, count) % 16 == 0 && offsetof(Sm, list) % 16 == 0 && offsetof(Sm, omass) % 16 == 0 &&
                  offsetof(Sm, omass_run) % 16 == 0 && offsetof(Sm, ocount) % 8 == 0 && offsetof(Sm, ocount_run) % 8 == 0 &&
                  offsetof(Sm, bmass) % 16 == 0 && offsetof(Sm, bcount) % 8 == 0 && sizeof(u64[kOctaves]) % 16 == 0,
              "read and written in pairs");
static_assert(2 * (sizeof(Sm) + 1024) <= 228 * 1024, "two CTAs to an SM");

// The CTA's state.  Functions take it from here, not as an argument: behind a pointer the compiler
// does not know that it is shared memory, and takes generic loads.
extern __shared__ __align__(16) unsigned char dynamic_smem[];
__device__ __forceinline__ Sm* state() { return reinterpret_cast<Sm*>(dynamic_smem); }

// The mass of a logit, and the weight of a token that counts (rare: not in line).
__device__ __noinline__ u64 mass_of(float l) {
  const Sm* const sm = state();
  const Scale sc = sm->row.scale;
  if (sc.wild && !(octaves_off(l, sc) < kFloorOctaves)) return 0;
  const Term x = term_of(fmaxf(l, sc.floor), sc, sm->table);
  return fixed_of(x.hi, x.lo);
}
// Whether min-p leaves it.  (What is past the floor counts as at the floor: a min-p below that leaves it
// among top-k's, behind all others and without mass, and the probabilities leave it out.)
__device__ __noinline__ bool min_p_keeps(float l) {
  const Sm* const sm = state();
  const Scale sc = sm->row.scale;
  if (sc.wild && !(octaves_off(l, sc) < kFloorOctaves)) return sm->row.min_p <= 0x1p-45f;
  return !below(term_of(fmaxf(l, sc.floor), sc, sm->table), sm->row.min_p);
}
__device__ __forceinline__ u64 weight_of(float l, int i, bool by_count) {
  const Sm* const sm = state();
  if (!sm->row.kept(l, i) || (sm->row.min_p > 0.f && !min_p_keeps(l))) return 0;
  return by_count ? 1 : mass_of(l);
}

// Running sums over the block of two values (the totals, too).
struct Two {
  u64 a, b;
};
__device__ __forceinline__ Two block_run(u64 a, u64 b, u64* part, Two* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    a += lane >= o ? x : 0;
    b += lane >= o ? y : 0;
  }
  __syncthreads();
  if (lane == 31) {
    part[warp] = a;
    part[kWarps + warp] = b;
  }
  __syncthreads();
  u64 x = part[lane % kWarps + (lane < kWarps ? 0 : kWarps)];      // lanes 0..15: a's parts, 16..31: b's
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    x += (lane & (kWarps - 1)) >= o ? y : 0;
  }
  const u64 pa = __shfl_sync(0xffffffffu, x, (warp + kWarps - 1) % kWarps), pb = __shfl_sync(0xffffffffu, x, kWarps + (warp + kWarps - 1) % kWarps);
  *total = Two{__shfl_sync(0xffffffffu, x, kWarps - 1), __shfl_sync(0xffffffffu, x, 31)};
  return Two{a + (warp ? pa : 0), b + (warp ? pb : 0)};
}
static_assert(kWarps == 16, "two sums over the warps in one");

__device__ __forceinline__ void clear_buckets(bool masses, bool carried) {
  Sm* const sm = state();
  for (int b = threadIdx.x; b < kBuckets; b += kThreads) {
    sm->count[b] = 0;
    if (masses) sm->limb[0][b] = sm->limb[1][b] = sm->limb[2][b] = 0;
    if (carried) sm->carried[b] = 0;
  }
}
template <int kOffset>
__device__ __forceinline__ void add_shared(uint32_t addr, unsigned v) {
  asm volatile("red.shared.add.u32 [%0+%2], %1;" ::"r"(addr), "r"(v), "n"(kOffset) : "memory");
}
// Into the bucket whose first limb is at `at`.  (Zeros too: a predicated addition to shared memory
// becomes a branch of three or four instructions, an addition takes 2.3 cycles of an SM's time.)
__device__ __forceinline__ void add_mass(uint32_t at, u64 m) {
  add_shared<0>(at, (unsigned)m & 0x7FFFu);
  add_shared<4 * kBuckets>(at, (unsigned)(m >> 15) & 0x7FFFu);
  add_shared<8 * kBuckets>(at, (unsigned)(m >> 30));
}

// A histogram pass over this CTA's tokens: put(eight logits, group).  Slices of more than
// kFlush tokens carry their limbs over on the way (a limb's sum stays below 2^31).
template <typename T, typename F>
__device__ __forceinline__ void histogram(const Row& r, F put) {
  Sm* const sm = state();
#pragma unroll 1
  for (int g = r.g0; g < r.g1; g += kFlush / kGroup) {
    r.each<T>(g, min(r.g1, g + kFlush / kGroup), put);
    if (r.carried) {
      __syncthreads();
      for (int b = threadIdx.x; b < kBuckets; b += kThreads) {
        sm->carried[b] += sm->limb[0][b] + ((u64)sm->limb[1][b] << 15) + ((u64)sm->limb[2][b] << 30);
        sm->limb[0][b] = sm->limb[1][b] = sm->limb[2][b] = 0;
      }
      __syncthreads();
    }
  }
}

// A branch on this is one that the compiler knows a warp's lanes to take together; within one on
// threadIdx.x / 32 a shuffle took 250 cycles.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// Running sums over the warp's lanes.  (Code that runs once waits for its instructions: a loop of
// thirty costs less than five copies of it.)
__device__ __forceinline__ void run_over_warp(u64& x, unsigned& y) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = 1; i < 32; i <<= 1) {
    const u64 px = __shfl_up_sync(0xffffffffu, x, i);
    const unsigned py = __shfl_up_sync(0xffffffffu, y, i);
    x += lane >= i ? px : 0;
    y += lane >= i ? py : 0;
  }
}

// After a histogram pass: the sums of each octave's buckets go to all CTAs, which keep the running
// ones over the CTAs.  The buckets stay where they are: of them one octave is looked at per
// border (all of them, summed up over the CTAs, took 2.5 to 7.5 us).
__device__ __forceinline__ unsigned ld_cluster(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
static_assert(offsetof(Sm, limb) == offsetof(Sm, count) + 4 * kBuckets, "the limbs follow the counts");
__device__ __forceinline__ u64 limbs_mass(unsigned a, unsigned b, unsigned c) { return a + ((u64)b << 15) + ((u64)c << 30); }
__device__ __noinline__ void share_octaves(bool masses, bool counts) {
  Sm* const sm = state();
  const int rank = sm->row.rank, size = sm->row.size, lane = threadIdx.x & 31, warp = warp_index();
  const bool carried = sm->row.carried;
  __syncthreads();
  // eight lanes to an octave, each every eighth bucket, from places whose banks differ within the warp
  constexpr int kLanes = 8;
  const int o = threadIdx.x / kLanes, k = threadIdx.x % kLanes;
  u64 w = 0;
  unsigned c = 0;
  if (o < kOctaves) {
#pragma unroll 2
    for (int i = 0; i < kPerOctave / kLanes; ++i) {
      const int b = o * kPerOctave + (i + o) % (kPerOctave / kLanes) * kLanes + k;
      if (masses) w += limbs_mass(sm->limb[0][b], sm->limb[1][b], sm->limb[2][b]);
      if (carried && masses) w += sm->carried[b];
      if (counts) c += sm->count[b];
    }
  }
#pragma unroll
  for (int i = kLanes / 2; i > 0; i >>= 1) {
    w += __shfl_xor_sync(0xffffffffu, w, i);
    c += __shfl_xor_sync(0xffffffffu, c, i);
  }
  if (o < kOctaves && k == 0) {
    sm->omass_run[o] = w;
    sm->ocount_run[o] = c;
  }
  __syncthreads();
  // a warp to a CTA: few and wide stores (every octave's to every CTA were 736 of one word)
  if (warp < size && lane < kOctaves / 2) {
    Sm* to = in_cta(sm, warp);
    *reinterpret_cast<ulonglong2*>(&to->omass[rank][2 * lane]) = *reinterpret_cast<const ulonglong2*>(&sm->omass_run[2 * lane]);
    *reinterpret_cast<uint2*>(&to->ocount[rank][2 * lane]) = *reinterpret_cast<const uint2*>(&sm->ocount_run[2 * lane]);
  }
  sm->row.barrier();
  if (warp == 0) {
    // octaves 2 lane and 2 lane + 1
    const int at = min(lane, kOctaves / 2 - 1);
    u64 x0 = 0, x1 = 0;
    unsigned y0 = 0, y1 = 0;
#pragma unroll
    for (int j = 0; j < kMaxCluster; ++j) {
      if (j >= size) break;
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&sm->omass[j][2 * at]);
      const uint2 y = *reinterpret_cast<const uint2*>(&sm->ocount[j][2 * at]);
      x0 += x.x; x1 += x.y;
      y0 += y.x; y1 += y.y;
    }
    x1 += x0;
    y1 += y0;
    u64 x = x1;
    unsigned y = y1;
    run_over_warp(x, y);
    if (lane < kOctaves / 2) {
      sm->omass_run[2 * lane] = x - x1 + x0;
      sm->omass_run[2 * lane + 1] = x;
      sm->ocount_run[2 * lane] = y - y1 + y0;
      sm->ocount_run[2 * lane + 1] = y;
    }
  }
  __syncthreads();
}
static_assert(kOctaves % 2 == 0 && kOctaves <= 64 && 8 * kOctaves <= kThreads, "two octaves to a lane");

// The buckets at which the running weight (counts or masses) reaches W0 and W1, each from 1 to
// the total: to found[0] and [1].  Every CTA looks it up for itself, in all CTAs' buckets (which
// stay as they are until the next histogram).
__device__ __noinline__ void find(u64 W0, u64 W1, bool by_count) {
  Sm* const sm = state();
  const int size = sm->row.size, lane = threadIdx.x & 31, warp = warp_index();
  const bool carried = sm->row.carried;
  __syncthreads();                           // (the last ones found are read)
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const u64 W = which ? W1 : W0;
    // (often both are in one bucket)
    if (which && W1 >= W0) {
      const Found f = sm->found[0];
      if (W1 - f.before <= (by_count ? (u64)f.count : f.mass)) {
        if (threadIdx.x == 0) sm->found[1] = f;
        __syncthreads();
        break;
      }
    }
    auto reached = [&](int o) { return o < kOctaves && (by_count ? (u64)sm->ocount_run[o] : sm->omass_run[o]) >= W; };
    const unsigned lo = __ballot_sync(0xffffffffu, reached(lane)), hi = __ballot_sync(0xffffffffu, reached(lane + 32));
    const int o = lo ? __ffs(lo) - 1 : hi ? 31 + __ffs(hi) : kOctaves - 1;
    // two warps to a CTA: few and wide loads
    const int k = warp / (kPerOctave / 32), b = threadIdx.x % kPerOctave;
    if (k < size) {
      const uint32_t at = ptx::map_to_cta(ptx::smem_addr(&sm->count[o * kPerOctave + b]), k);
      const unsigned c = ld_cluster(at);
      u64 w = limbs_mass(ld_cluster(at + 4 * kBuckets), ld_cluster(at + 8 * kBuckets), ld_cluster(at + 12 * kBuckets));
      if (carried) w += in_cta(sm, k)->carried[o * kPerOctave + b];
      sm->bmass[k][b] = w;
      sm->bcount[k][b] = c;
    }
    __syncthreads();
    if (warp == 0) {
      u64 w0 = 0, w1 = 0;
      unsigned c0 = 0, c1 = 0;
#pragma unroll
      for (int j = 0; j < kMaxCluster; ++j) {
        if (j >= size) break;
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&sm->bmass[j][2 * lane]);
        const uint2 c = *reinterpret_cast<const uint2*>(&sm->bcount[j][2 * lane]);
        w0 += w.x; w1 += w.y;
        c0 += c.x; c1 += c.y;
      }
      u64 x = w0 + w1;
      unsigned y = c0 + c1;
      run_over_warp(x, y);
      const u64 m_end = (o ? sm->omass_run[o - 1] : 0) + x;
      const unsigned c_end = (o ? sm->ocount_run[o - 1] : 0) + y;
      const u64 m_mid = m_end - w1, m_begin = m_mid - w0;
      const unsigned c_mid = c_end - c1, c_begin = c_mid - c0;
      const u64 begin = by_count ? c_begin : m_begin, mid = by_count ? c_mid : m_mid, end = by_count ? c_end : m_end;
      const int first = o * kPerOctave + 2 * lane;
      if (begin < W && mid >= W) sm->found[which] = Found{begin, m_begin, w0, first, c0};
      if (mid < W && end >= W) sm->found[which] = Found{mid, m_mid, w1, first + 1, c1};
    }
    __syncthreads();
  }
}
static_assert(kThreads == kPerOctave * kMaxCluster, "a thread for each CTA's part of an octave's buckets");

// The tokens for which like(logit) and then want(logit, index) hold, collected by the
// first CTA; returns how many there are (to all CTAs), more than kList are not collected.
template <typename T, typename L, typename F>
__device__ __forceinline__ int gather(const Row& r, L like, F want) {
  Sm* const sm = state();
  if (threadIdx.x == 0) sm->n = 0;
  __syncthreads();
  r.each<T>(r.g0, r.g1, [&](const float (&v)[kGroup], int g) {
    unsigned hit = 0;
#pragma unroll
    for (int e = 0; e < kGroup; ++e) hit |= like(v[e]) ? 1u << e : 0u;
#pragma unroll 1
    for (; hit; hit &= hit - 1) {
      const int i = kGroup * g + __ffs(hit) - 1;
      if (i >= r.V) break;
      const float l = r.clean(entry(static_cast<const T*>(r.logits), i));
      const uint32_t key = key_of(l);
      if (key && want(l, i)) {
        const unsigned at = atomicAdd(&sm->n, 1u);
        if (at < kList) sm->pick[at] = ((u64)key << 32) | (uint32_t)~i;
      }
    }
  });
  __syncthreads();
  if (threadIdx.x < r.size) in_cta(sm, threadIdx.x)->picked[r.rank] = sm->n;
  r.barrier();
  int n = 0;
  for (int k = 0; k < r.size; ++k) n += sm->picked[k];
  if (n <= kList && r.rank == 0) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      int k = 0, j = i;                // the j-th of CTA k's
      for (; j >= (int)sm->picked[k]; ++k) j -= sm->picked[k];
      sm->list[i] = in_cta(sm, k)->pick[j];
    }
  }
  r.barrier();       // the picked tokens are read, and may be picked anew
  if (r.trigger) pdl_trigger();
  return n;
}

__device__ __forceinline__ uint32_t entry_key(u64 e) { return (uint32_t)(e >> 32); }
__device__ __forceinline__ int entry_index(u64 e) { return (int)~(uint32_t)e; }

// The list in the tokens' order, and their running masses (0 for what min-p leaves out).
__device__ __noinline__ void sort_list(int n) {
  Sm* const sm = state();
  const int tid = threadIdx.x;
  const bool by_min_p = sm->row.min_p > 0.f;
  auto mass_at = [&](int i) {
    const float l = value_of(entry_key(sm->list[i]));
    return by_min_p && !min_p_keeps(l) ? 0 : mass_of(l);
  };
  __syncthreads();
  if (n <= kThreads / 4) {
    // each token's place is how many stand before it, and its sum theirs and its own; four threads
    // count for a token
    u64* const mass = sm->pick;
    if (tid < n) mass[tid] = mass_at(tid);
    if (tid < 8) sm->list[n + tid] = mass[n + tid] = 0;
    __syncthreads();
    u64 mine = 0, run = 0;
    int place = 0;
    const int i = tid >> 2, quarter = (n + 7) / 8 * 2, from = (tid & 3) * quarter, to = from + quarter;
    if (i < n) {
      mine = sm->list[i];
      for (int k = from; k < to; k += 2) {       // (zeros past the list: from and to are even)
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sm->list + k), m = *reinterpret_cast<const ulonglong2*>(mass + k);
        place += (x.x > mine) + (x.y > mine);
        run += (x.x >= mine ? m.x : 0) + (x.y >= mine ? m.y : 0);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      place += __shfl_xor_sync(0xffffffffu, place, o);
      run += __shfl_xor_sync(0xffffffffu, run, o);
    }
    __syncthreads();
    if (i < n && (tid & 3) == 0) {
      sm->list[place] = mine;
      sm->sum[place] = run;
    }
    __syncthreads();
    return;
  }
  u64 e[2], m[2];                                  // two tokens to a thread
  uint32_t top = 0, low = ~0u;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * tid + j;
    e[j] = i < n ? sm->list[i] : 0;
    m[j] = i < n ? mass_at(i) : 0;
    if (i < n) {
      top = max(top, entry_key(e[j]));
      low = min(low, entry_key(e[j]));
    }
  }
  // Parts of the keys' range, their counts and first places; in a part each token counts what
  // stands before it.  Parts of many (equal keys) are left to a sorting network.
  unsigned* const count = reinterpret_cast<unsigned*>(sm->pick);
  unsigned* const first = count + kList;
  count[tid] = count[tid + kThreads] = 0;
  if (tid == 0) {
    sm->khi = 0;
    sm->klo = ~0u;
  }
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, top);
  low = __reduce_min_sync(0xffffffffu, low);
  if ((tid & 31) == 0) {
    atomicMax(&sm->khi, top);
    atomicMin(&sm->klo, low);
  }
  __syncthreads();
  top = sm->khi;
  const int shift = max(0, 32 - __clz(top - sm->klo) - 10);      // (kList parts)
  unsigned part[2], slot[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    part[j] = (top - entry_key(e[j])) >> shift;
    if (e[j]) slot[j] = atomicAdd(&count[part[j]], 1u);
  }
  __syncthreads();
  const unsigned c0 = count[2 * tid], c1 = count[2 * tid + 1];
  Two total;
  if (!__syncthreads_or(c0 > 32 || c1 > 32)) {
    const unsigned upto = (unsigned)block_run(c0 + c1, 0, sm->part, &total).a;
    first[2 * tid] = upto - c1 - c0;
    first[2 * tid + 1] = upto - c1;
    __syncthreads();
    unsigned place[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (e[j]) sm->sum[first[part[j]] + slot[j]] = e[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      place[j] = 0;
      if (!e[j]) continue;
      place[j] = first[part[j]];
      const u64* const others = sm->sum + place[j];
      for (unsigned k = count[part[j]]; k > 0; --k) place[j] += others[k - 1] > e[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (!e[j]) continue;
      sm->list[place[j]] = e[j];
      sm->sum[place[j]] = m[j];
    }
    __syncthreads();
    m[0] = 2 * tid < n ? sm->sum[2 * tid] : 0;
    m[1] = 2 * tid + 1 < n ? sm->sum[2 * tid + 1] : 0;
  } else {
    for (int i = n + tid; i < kList; i += kThreads) sm->list[i] = 0;
    for (int len = 2; len <= kList; len *= 2) {
      for (int step = len / 2; step > 0; step /= 2) {
        __syncthreads();
        const int i = 2 * step * (tid / step) + tid % step;      // kThreads pairs (i, i + step)
        const u64 a = sm->list[i], b = sm->list[i + step];
        if ((a < b) == ((i & len) == 0)) {
          sm->list[i] = b;
          sm->list[i + step] = a;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) m[j] = 2 * tid + j < n ? mass_at(2 * tid + j) : 0;
  }
  const u64 end = block_run(m[0] + m[1], 0, sm->part, &total).a;
  sm->sum[2 * tid] = end - m[1];
  sm->sum[2 * tid + 1] = end;
  __syncthreads();
}
static_assert(kList == 1024, "ten bits of a part");
static_assert(kList == 2 * kThreads, "two tokens of the list for each thread");

// The first place of the list at which the running mass reaches W (the last one of n if none does).
__device__ __noinline__ int place_in_list(int n, u64 W) {
  Sm* const sm = state();
  if (threadIdx.x == 0) sm->at = n - 1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (sm->sum[i] >= W && (i == 0 || sm->sum[i - 1] < W)) sm->at = i;
  __syncthreads();
  const int at = sm->at;
  __syncthreads();
  return at;
}
__device__ __forceinline__ void tell_border(const Border& b) {
  Sm* const sm = state();      // one thread
  for (int k = 0; k < sm->row.size; ++k) in_cta(sm, k)->border = b;
}

// Counts and masses of the buckets (of tokens that min-p leaves: kMinP where it is on).
template <typename T, bool kMinP>
__device__ __noinline__ void bucket_masses(bool cleared, bool counts) {
  Sm* const sm = state();
  const Row r = sm->row;
  if (!cleared) {
    clear_buckets(true, r.carried);
    __syncthreads();
  }
  const uint32_t limbs = ptx::smem_addr(sm->limb), counts_at = ptx::smem_addr(sm->count);
  if (r.scale.wild) {
    histogram<T>(r, [&](const float (&v)[kGroup], int) {
      for (int e = 0; e < kGroup; ++e) {
        if (!(v[e] > -INFINITY) || (kMinP && !min_p_keeps(v[e]))) continue;
        add_mass(limbs + 4 * bucket_of(v[e], r.scale), mass_of(v[e]));
        if (counts) add_shared<0>(counts_at + 4 * bucket_of(v[e], r.scale), 1);
      }
    });
    share_octaves(true, counts);
    return;
  }
  histogram<T>(r, [&](const float (&v)[kGroup], int) {
    // (four at a time: eight do not leave the registers for it)
#pragma unroll
    for (int e0 = 0; e0 < kGroup; e0 += 4) {
      u64 m[4];
      uint32_t at[4];
      bool in[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const Term x = term_of(fmaxf(v[e0 + e], r.scale.floor), r.scale, sm->table);
        m[e] = fixed_of(x.hi, x.lo);
        at[e] = 4 * (x.place / (kTable / kPerOctave));       // + kBase
        in[e] = !kMinP || !below(x, r.min_p);
        if (kMinP && !in[e]) m[e] = 0;
      }
      constexpr uint32_t kBase = 4 * (kMagicBits / (kTable / kPerOctave));
#pragma unroll
      for (int e = 0; e < 4; ++e)       // (what has no mass goes to the lane's own place, not all of it to one)
        add_mass(at[e] < kBase + 4 * kMassBuckets ? limbs - kBase + at[e] : limbs + 4 * (threadIdx.x & 31), m[e]);
      if (counts) {
#pragma unroll
        for (int e = 0; e < 4; ++e) add_shared<0>(counts_at - kBase + at[e], v[e0 + e] > -INFINITY && in[e]);
      }
    }
  });
  share_octaves(true, counts);
}

template <typename T>
__device__ __forceinline__ void row_masses(bool cleared, bool counts) {
  if (state()->row.min_p > 0.f) bucket_masses<T, true>(cleared, counts); else bucket_masses<T, false>(cleared, counts);
}

// The token at which the running weight reaches W (the rows of buckets as share_octaves left
// them): to sm->border of all CTAs.  Returns whether they are still those of the whole row.
template <typename T>
__device__ __noinline__ bool locate(u64 W, bool by_count) {
  Sm* const sm = state();
  const Row r = sm->row;
  const T* logits = static_cast<const T*>(r.logits);
  bool whole = true;
  find(W, W, by_count);
  const int bucket = sm->found[0].bucket;
  u64 before = sm->found[0].before, mass_before = sm->found[0].mass_before;
  auto counts = [&](float l, int i) { return weight_of(l, i, by_count) > 0; };
  const Range range = range_of(bucket, bucket, r.scale);
  int n = gather<T>(r, [&](float l) { return range.has(l); },
                    [&](float l, int i) { return bucket_of(l, r.scale) == bucket && counts(l, i); });
  if (n > kList) {
    // The bucket's keys: [klo, khi], by bisection (a larger key is in the same bucket or one before).
    if (threadIdx.x < 2) {
      const int j = bucket - threadIdx.x;              // thread 0: the first key in bucket j or before; 1: in j - 1
      uint32_t lo = 0x00800000u, hi = key_of(r.scale.max) + 1;      // from the lowest finite value
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (bucket_of(value_of(mid), r.scale) <= j) hi = mid; else lo = mid + 1;
      }
      if (threadIdx.x == 0) sm->klo = lo; else sm->khi = lo - 1;
    }
    __syncthreads();
    uint32_t klo = sm->klo, khi = sm->khi;
    auto among = [&](float l) {
      const uint32_t key = key_of(l);
      return key >= klo && key <= khi;
    };
    while (n > kList && klo < khi) {
      int shift = 0;
      while (((khi - klo) >> shift) >= kBuckets) ++shift;
      clear_buckets(true, r.carried);
      __syncthreads();
      histogram<T>(r, [&](const float (&v)[kGroup], int g) {
#pragma unroll 1
        for (int e = 0; e < kGroup; ++e) {
          const float l = kGroup * g + e < r.V ? r.clean(entry(logits, kGroup * g + e)) : -INFINITY;
          const uint32_t key = key_of(l);
          if (key < klo || key > khi) continue;
          const u64 w = weight_of(l, kGroup * g + e, by_count);
          if (w == 0) continue;
          const int b = (int)((khi - key) >> shift);
          const u64 m = by_count ? mass_of(l) : w;
          add_mass(ptx::smem_addr(&sm->limb[0][b]), m);
          if (by_count) atomicAdd(&sm->count[b], 1u);
        }
      });
      share_octaves(true, by_count);
      whole = false;
      find(W - before, W - before, by_count);
      before += sm->found[0].before;
      mass_before += sm->found[0].mass_before;
      khi -= (uint32_t)sm->found[0].bucket << shift;
      const uint32_t width = (1u << shift) - 1;
      if (khi - klo > width) klo = khi - width;
      n = gather<T>(r, among, counts);
    }
    if (n > kList) {
      // One key is left: its tokens in index order.
      const float l = value_of(klo);
      const u64 m = mass_of(l), each = by_count ? 1 : m;
      u64 q = (W - before + each - 1) / each;          // the q-th of them
      const u64 upto = mass_before + q * m;
      int owner = 0;
      for (int k = 0; k < r.size; ++k) {               // (gather told how many each CTA has)
        owner = k;
        if (sm->picked[k] >= q) break;
        q -= sm->picked[k];
      }
      if (owner == r.rank) {
        u64 done = 0;
        for (int g = r.g0; g < r.g1; g += kThreads) {
          float v[kGroup];
          unsigned hit = 0;
          if (g + (int)threadIdx.x < r.g1) {
            load8(logits, g + threadIdx.x, r.V, v);
#pragma unroll
            for (int e = 0; e < kGroup; ++e) {
              const int i = kGroup * (g + threadIdx.x) + e;
              hit |= (unsigned)(key_of(r.clean(v[e])) == klo && r.kept(l, i)) << e;
            }
          }
          Two total;
          const u64 mine = __popc(hit), run = done + block_run(mine, 0, sm->part, &total).a;
          if (run >= q && run - mine < q) {
            for (u64 k = run - mine + 1; k < q; ++k) hit &= hit - 1;
            tell_border(Border{upto, klo, kGroup * (g + (int)threadIdx.x) + __ffs(hit) - 1});
          }
          done += total.a;
          if (done >= q) break;
        }
      }
      r.barrier();
      return whole;
    }
  }
  if (r.rank == 0) {
    sort_list(n);
    const int at = by_count ? (int)(W - before) - 1 : place_in_list(n, W - before);
    if (threadIdx.x == 0)
      tell_border(Border{mass_before + sm->sum[at], entry_key(sm->list[at]), entry_index(sm->list[at])});
  }
  r.barrier();
  return whole;
}

// Probabilities of eight tokens
__device__ __forceinline__ void store8(float* row, int g, int V, const float (&v)[kGroup]) {
  const int x = kGroup * g;
  if (x + kGroup <= V) {
    *reinterpret_cast<float4*>(row + x) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(row + x + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    for (int e = 0; x + e < V; ++e) row[x + e] = v[e];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* row, int g, int V, const float (&v)[kGroup]) {
  const int x = kGroup * g;
  if (x + kGroup <= V) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(row + x) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    for (int e = 0; x + e < V; ++e) row[x + e] = __float2bfloat16_rn(v[e]);
  }
}

// The last token left, as locate or the first CTA told it, becomes the cut; its mass is returned.
__device__ __forceinline__ u64 take_cut() {
  Sm* const sm = state();
  const Border b = sm->border;
  __syncthreads();
  if (threadIdx.x == 0) {
    sm->row.cut = value_of(b.key);
    sm->row.cut_index = b.index;
  }
  __syncthreads();
  return b.mass;
}

// The last bucket of those, from the first on, in which `quota` of this CTA's threads have their
// largest logit (counted in the buckets); the largest of the CTAs'.  kBuckets: some CTA has fewer.
__device__ __noinline__ int bucket_limit(int quota) {
  Sm* const sm = state();
  const int lane = threadIdx.x & 31, warp = warp_index(), size = sm->row.size;
  __syncthreads();
  const unsigned* const count = sm->count;
  constexpr int kLanes = 8;                  // as in share_octaves
  const int o = threadIdx.x / kLanes;
  unsigned c = 0;
  if (o < kOctaves) {
#pragma unroll
    for (int i = 0; i < kPerOctave / kLanes; ++i)
      c += count[o * kPerOctave + (i + o) % (kPerOctave / kLanes) * kLanes + threadIdx.x % kLanes];
  }
#pragma unroll
  for (int i = kLanes / 2; i > 0; i >>= 1) c += __shfl_xor_sync(0xffffffffu, c, i);
  if (o < kOctaves && threadIdx.x % kLanes == 0) sm->ocount_run[o] = c;
  __syncthreads();
  if (warp == 0) {
    auto run = [&](unsigned y) {
#pragma unroll 1
      for (int i = 1; i < 32; i <<= 1) {
        const unsigned py = __shfl_up_sync(0xffffffffu, y, i);
        y += lane >= i ? py : 0;
      }
      return y;
    };
    const uint2 y = lane < kOctaves / 2 ? *reinterpret_cast<const uint2*>(&sm->ocount_run[2 * lane]) : make_uint2(0, 0);
    const unsigned end = run(y.x + y.y), at = __ballot_sync(0xffffffffu, end >= (unsigned)quota);
    int bucket = kBuckets;
    if (at) {
      // of the first pair of octaves, bucket by bucket (four to a lane)
      const int pair = __ffs(at) - 1;
      const unsigned left = quota - (__shfl_sync(0xffffffffu, end, pair) - __shfl_sync(0xffffffffu, y.x + y.y, pair));
      const int b = 2 * kPerOctave * pair + 4 * lane;
      const uint4 n = *reinterpret_cast<const uint4*>(&count[b]);
      const unsigned upto = run(n.x + n.y + n.z + n.w), before = upto - (n.x + n.y + n.z + n.w);
      const int first = __ffs(__ballot_sync(0xffffffffu, upto >= left)) - 1;
      const int mine = b + (before + n.x >= left ? 0 : before + n.x + n.y >= left ? 1 : before + n.x + n.y + n.z >= left ? 2 : 3);
      bucket = __shfl_sync(0xffffffffu, mine, first);
    }
    if (lane < size) in_cta(sm, lane)->limit[sm->row.rank] = bucket;
  }
  sm->row.barrier();
  int bucket = sm->limit[0];
  for (int k = 1; k < size; ++k) bucket = max(bucket, sm->limit[k]);
  return bucket;
}
static_assert(2 * kPerOctave == 4 * 32 && kOctaves % 2 == 0, "two octaves' buckets, four to a lane");

// Few tokens are left by top-k (k > 0) or min-p: the first CTA sorts them.  False where there
// are more than it can sort.  Where k threads have a largest logit (`mine`) in some bucket or one before,
// the k likeliest tokens are there, and not many others; a bucket in which each of the CTAs has
// its share of k threads is soon found.  What min-p leaves is there by its value.
template <typename T>
__device__ __noinline__ bool few_tokens(float mine, int k, float min_p, float p, float u, int32_t* token, bool probs) {
  Sm* const sm = state();
  const Row r = sm->row;
  int last_bucket = kBuckets;         // (all)
  if (k > 0 && k <= kList / 2) {
    mine = r.clean(mine);
    if (mine > -INFINITY) atomicAdd(&sm->count[bucket_of(mine, r.scale)], 1u);
    last_bucket = bucket_limit((k + r.size - 1) / r.size);
    if (last_bucket == kBuckets) {           // (a CTA's slice may be masked)
      share_octaves(false, true);
      const unsigned threads = sm->ocount_run[kOctaves - 1];
      if (threads >= (unsigned)k) {
        find((u64)k, (u64)k, true);
        last_bucket = sm->found[0].bucket;
      }
    }
  }
  // (a bucket's bounds are off by half a place, a 32nd of it)
  if (min_p > 0.f) last_bucket = min(last_bucket, (int)(-log2f(min_p) * kPerOctave) + 1);
  const Range range = range_of(0, last_bucket, r.scale);
  const int n = gather<T>(r, [&](float l) { return range.has(l); },
                          [&](float l, int) { return bucket_of(l, r.scale) <= last_bucket; });
  if (n > kList) return false;
  if (r.rank == 0) {
    sort_list(n);
    const int left = k > 0 ? min(k, n) : n;
    const u64 Z = sm->sum[left - 1];
    // (without top-p the list's tokens that min-p leaves out are behind the last one of those left, and add nothing)
    const int last = p < 1.f ? place_in_list(left, reach(p, Z)) : left - 1;
    const u64 M = sm->sum[last];
    const int at = token ? place_in_list(left, pass(u, M)) : 0;
    if (threadIdx.x == 0) {
      if (token) *token = entry_index(sm->list[at]);
      if (probs) tell_border(Border{M, entry_key(sm->list[last]), entry_index(sm->list[last])});
    }
  }
  if (probs) r.barrier();
  return true;
}

// Top-p's border and the token at once: the sum that top-p leaves of Z lies within the bucket of
// its border, so that the token's bucket is known but for one or two.  False where there are
// more tokens than the first CTA can sort.
template <typename T>
__device__ __noinline__ bool both(u64 Z, float p, float u, int32_t* token, bool probs) {
  Sm* const sm = state();
  const Row r = sm->row;
  const u64 W = reach(p, Z);
  find(W, W, false);
  const int bucket = sm->found[0].bucket;
  const u64 before = sm->found[0].before, upto = before + sm->found[0].mass;
  find(pass(u, W), pass(u, upto), false);
  const int b0 = sm->found[0].bucket, b1 = sm->found[1].bucket;
  const u64 t_before = sm->found[0].before;
  // The list's running masses go from the token's first bucket on; the border's are `apart` behind
  // them where there are other buckets between.
  const u64 apart = bucket > b1 ? before - (sm->found[1].before + sm->found[1].mass) : 0;
  const Range border = range_of(bucket, bucket, r.scale), inner = range_of(b0, b1, r.scale);
  const int n = gather<T>(r, [&](float l) { return border.has(l) || inner.has(l); }, [&](float l, int i) {
    const int b = bucket_of(l, r.scale);
    return (b == bucket || (b >= b0 && b <= b1)) && weight_of(l, i, false) > 0;
  });
  if (n > kList) return false;
  if (r.rank == 0) {
    sort_list(n);
    const int last = place_in_list(n, W - t_before - apart);
    const u64 M = t_before + apart + sm->sum[last];
    const int at = place_in_list(n, pass(u, M) - t_before);
    if (threadIdx.x == 0) {
      *token = entry_index(sm->list[at]);
      if (probs) tell_border(Border{M, entry_key(sm->list[last]), entry_index(sm->list[last])});
    }
  }
  if (probs) r.barrier();
  return true;
}

// Rows whose cuts may lie anywhere; returns the sum that is left.
template <typename T>
__device__ __noinline__ u64 many(bool cleared, int k, float p, float u, int32_t* token, bool probs) {
  Sm* const sm = state();
  row_masses<T>(cleared, k > 0);
  const int rank = sm->row.rank;
  u64 M = sm->omass_run[kOctaves - 1];
  const u64 all = sm->ocount_run[kOctaves - 1];
  if (k > 0 && (u64)k < all) {
    const bool whole = locate<T>((u64)k, true);
    M = take_cut();
    if (!whole) row_masses<T>(false, false);
  }
  bool whole = true;
  if (p < 1.f) {
    if (token && both<T>(M, p, u, token, probs)) return probs ? take_cut() : 0;
    whole = locate<T>(reach(p, M), false);
    M = take_cut();
  }
  if (token) {
    if (!whole) row_masses<T>(false, false);
    locate<T>(pass(u, M), false);
    if (threadIdx.x == 0 && rank == 0) *token = sm->border.index;
  }
  return M;
}

// Rows that few_tokens takes.  (A list for min-p that turns out too long costs 3 us, one that does not saves 15.)
__device__ __forceinline__ bool few_left(float temperature, int k, float min_p) {
  return temperature == 0.f || (k > 0 && k <= kList / 2) || min_p >= 0x1p-10f;
}

// The row of this cluster.  CTAs get an SM of their own while there is one, and share it from then on:
// the rows with a histogram of masses come first (of up to kThreads rows), so that they share their
// SMs with others.
__device__ __forceinline__ int row_in_order(const SampleCall& c, int at) {
  Sm* const sm = state();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = at / kThreads * kThreads, i = first + threadIdx.x;
  const bool in = i < c.N;
  const bool late = in && few_left(c.temperature ? c.temperature[i] : 1.f, c.top_k ? c.top_k[i] : 0, c.min_p ? c.min_p[i] : 0.f);
  const unsigned lates = __ballot_sync(0xffffffffu, late), soons = __ballot_sync(0xffffffffu, in && !late);
  if (lane == 0) sm->part[warp] = __popc(soons) | (u64)__popc(lates) << 32;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const u64 n = sm->part[k];
    before += k < warp ? n : 0;
    all += n;
  }
  const unsigned below = (1u << lane) - 1;
  const int place = late ? (int)(unsigned)all + (int)(before >> 32) + __popc(lates & below)
                         : (int)(unsigned)before + __popc(soons & below);
  if (in && place == at - first) sm->at = i;
  __syncthreads();
  return sm->at;
}

template <typename T, typename P>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleCall c, int size, bool crowded, bool ordered, int* status) {
  Sm* const sm = state();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 64) sm->roots[tid] = power_of_roots(tid < 32 ? tid : 32 * (tid - 32));
  __syncthreads();
  for (int j = tid; j < kTable; j += kThreads) {
    const float2 low = sm->roots[j % 32];
    sm->table[j] = table_entry(times(sm->roots[32 + j / 32], low.x, low.y), j);
  }
  Row r;
  r.size = size;
  r.rank = size > 1 ? (int)ptx::cluster_ctarank() : 0;
  r.barrier();             // the cluster's CTAs run: their shared memory may be written
  pdl_wait();
  r.trigger = crowded && !c.probs;
  if (!crowded) pdl_trigger();
  const int row = ordered ? row_in_order(c, blockIdx.x / size) : blockIdx.x / size;
  r.logits = static_cast<const T*>(c.logits) + (size_t)row * c.row_stride;
  r.V = c.V;
  const int groups = (c.V + kGroup - 1) / kGroup, per = (groups + size - 1) / size;
  r.g0 = min(groups, r.rank * per);
  r.g1 = min(groups, r.g0 + per);
  r.carried = per > kFlush / kGroup;
  // (asked for ahead of the first pass)
  const float temp = c.temperature ? c.temperature[row] : 1.f;
  float mp = c.min_p ? c.min_p[row] : 0.f;
  const int top_k = c.top_k ? c.top_k[row] : 0;
  const float p = c.top_p ? c.top_p[row] : 1.f;
  float u = c.tokens ? c.u[row] : 0.f;
  u = u >= 1.f ? 1.f - 0x1p-24f : u;                 // (NaN stays, and counts as 0: fraction)
  // What goes by the settings alone, and the buckets' clearing, while the logits are on their way.
  const bool greedy = temp == 0.f;
  constexpr double kLog2e = 1.4426950408889634074;
  constexpr float kLog2eHigh = (float)kLog2e, kLog2eLow = (float)(kLog2e - (double)kLog2eHigh);
  const float2 scale = pair_divide(kLog2eHigh, kLog2eLow, greedy ? 1.f : temp, 0.f);
  r.scale.ch = fminf(scale.x, 3.4028234e38f);
  r.scale.cl = scale.x > 0.f && scale.x < 3.4028234e38f ? scale.y : 0.f;     // (temperatures of 0x1p-128, infinity)
  const float off = kFloorOctaves / r.scale.ch;
  mp = mp > 0.f ? fminf(mp, 1.f) : 0.f;
  r.min_p = mp;
  const int k = greedy ? 1 : top_k;
  const bool few = few_left(temp, top_k, mp);
  clear_buckets(!few, r.carried && !few);
  r.infinite = false;
  float mine = -INFINITY;         // this thread's largest logit (fmaxf passes over NaN)
  r.each<T>(r.g0, r.g1, [&](const float (&v)[kGroup], int) {
#pragma unroll
    for (int e = 0; e < kGroup; ++e) mine = fmaxf(mine, v[e]);
  });
  float m = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sm->fpart[warp] = m;
  __syncthreads();
  m = sm->fpart[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (tid < size) in_cta(sm, tid)->max[r.rank] = m;
  r.barrier();
  m = sm->max[0];
  for (int k = 1; k < size; ++k) m = fmaxf(m, sm->max[k]);
  P* probs = c.probs ? static_cast<P*>(c.probs) + (size_t)row * c.probs_stride : nullptr;
  int32_t* token = c.tokens ? c.tokens + row : nullptr;
  const bool bad = !(temp >= 0.f);
  if (bad || m == -INFINITY) {
    if (tid == 0 && r.rank == 0) {
      if (bad) report(status);
      if (token) *token = -1;
    }
    const float zero[kGroup] = {};
    if (probs)
      for (int g = r.g0 + tid; g < r.g1; g += kThreads) store8(probs, g, c.V, zero);
    return;
  }
  r.infinite = m == INFINITY;
  r.scale.max = r.infinite ? 0.f : m;
  const float ulp = __uint_as_float((__float_as_uint(r.scale.max) & 0x7F800000u)) * 0x1p-23f;
  r.scale.wild = !(r.scale.ch * ulp <= 0.0625f && off < 1e36f && fabsf(r.scale.max) < 1e36f);
  r.scale.floor = r.scale.wild ? -3.4028234e38f : __fsub_rd(r.scale.max, off);
  r.cut = -INFINITY;
  r.cut_index = INT_MAX;
  if (tid == 0) sm->row = r;
  __syncthreads();
  u64 M = 0;
  if (few && few_tokens<T>(mine, k, mp, p, u, token, probs != nullptr)) {
    if (probs) M = take_cut();
  } else {
    M = many<T>(!few, k, p, u, token, probs != nullptr);
  }
  if (!probs) return;
  const Row row_now = sm->row;
  const Scale sc = row_now.scale;
  const float Mh = __ull2float_rn(M);
  const float2 inv = pair_divide((float)(1ull << kMassBits), 0.f, Mh, (float)(long long)(M - __float2ull_rn(Mh)));
  const float low = sc.wild ? -INFINITY : __fsub_rd(sc.max, 60.0001f / sc.ch);      // below: 0
  row_now.each<T>(row_now.g0, row_now.g1, [&](const float (&v)[kGroup], int g) {
    float out[kGroup];
    unsigned left = 0, last = 0;
#pragma unroll
    for (int e = 0; e < kGroup; ++e) {
      out[e] = 0.f;
      left |= v[e] >= row_now.cut && v[e] > low ? 1u << e : 0u;
      last |= v[e] == row_now.cut ? 1u << e : 0u;
    }
    if (last & left) {         // of tokens like the last one those up to it
      const int upto = row_now.cut_index - kGroup * g;
      left &= ~last | (upto < 0 ? 0u : upto < kGroup ? (2u << upto) - 1 : ~0u);
    }
    if (sc.wild) {
#pragma unroll 1
      for (int e = 0; e < kGroup; ++e)
        if (!(octaves_off(v[e], sc) < 60.f)) left &= ~(1u << e);
    }
    if (row_now.min_p > 0.f) {
#pragma unroll 1
      for (unsigned x = left; x; x &= x - 1) {
        const int e = __ffs(x) - 1;
        if (below(term_of(row_now.clean(entry(static_cast<const T*>(row_now.logits), kGroup * g + e)), sc, sm->table), row_now.min_p))
          left &= ~(1u << e);
      }
    }
    if (left) {
      // e / M rounded once: the pair times 2^44 / M as a pair
#pragma unroll
      for (int e = 0; e < kGroup; ++e) {
        const Term x = term_of(left >> e & 1u ? v[e] : sc.max, sc, sm->table);
        const float q = fmaf(x.hi, inv.x, fmaf(x.hi, inv.y, x.lo * inv.x));
        out[e] = left >> e & 1u ? q : 0.f;
      }
    }
    store8(probs, g, c.V, out);
  });
}

void cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&attr)[2], int clusters, int size, cudaStream_t st) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3((unsigned)(clusters * size));
  cfg->blockDim = dim3(kThreads);
  cfg->dynamicSmemBytes = sizeof(Sm);
  cfg->stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// The shared-memory opt-in, once per device (setting it twice is harmless).
bool set_attributes() {
  static std::atomic<bool> done[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (done[dev].load(std::memory_order_acquire)) return true;
  auto allow = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Sm)) == cudaSuccess;
  };
  if (!allow(sample_kernel<float, float>) || !allow(sample_kernel<float, __nv_bfloat16>) ||
      !allow(sample_kernel<__nv_bfloat16, float>) || !allow(sample_kernel<__nv_bfloat16, __nv_bfloat16>))
    return false;
  done[dev].store(true, std::memory_order_release);
  return true;
}

// CTAs per row: as many as leave all N clusters resident at once.
int cluster_size(int N) {
  // Filled on first use per device; concurrent first calls compute and store the same values.
  static std::atomic<int> resident[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  for (int size = kMaxCluster; size > 1; --size) {
    int n = resident[dev][size].load(std::memory_order_relaxed);
    if (n == 0) {
      cudaLaunchConfig_t cfg;
      cudaLaunchAttribute attr[2];
      cluster_config(&cfg, attr, 64, size, nullptr);
      if (cudaOccupancyMaxActiveClusters(&n, sample_kernel<float, float>, &cfg) != cudaSuccess || n <= 0) n = -1;
      resident[dev][size].store(n, std::memory_order_relaxed);
    }
    if (n >= N) return size;
  }
  return 1;
}

}  // namespace

cudaError_t launch_sample(const SampleCall& c, cudaStream_t st) {
  int* status = bmm_status_ptr();
  if (!status || !set_attributes()) return cudaErrorInvalidValue;
  const int size = cluster_size(c.N);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  cluster_config(&cfg, attr, c.N, size, st);
  // Where every CTA has an SM of its own the order of the rows is of no use, and the next kernel's CTAs
  // may come at once.  Where not, those that come while this one's leave are put wherever there is
  // room, several to an SM while others idle (64 mixed rows 50 us in place of 37, 96 with probabilities 67 of 50).
  const bool crowded = (long long)c.N * size > mla_device_sm_count();
  const bool ordered = crowded && (c.temperature || c.top_k || c.min_p);
  auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, c, size, crowded, ordered, status); };
  if (c.bf16)
    return c.probs_bf16 ? launch(sample_kernel<__nv_bfloat16, __nv_bfloat16>) : launch(sample_kernel<__nv_bfloat16, float>);
  return c.probs_bf16 ? launch(sample_kernel<float, __nv_bfloat16>) : launch(sample_kernel<float, float>);
}

}  // namespace mla
