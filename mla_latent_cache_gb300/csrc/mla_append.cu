// New tokens' queries and cache rows: per-head query norm, latent norm, position
// rotation and the write into the paged cache, in one pass.
//
// For token i, head h, with q the 192-wide query row [nope 128 | rope 64] and kv the
// 576-wide row [latent 512 | rope 64]:
//   q'   = q / sqrt(mean(q^2) + eps) * w_q     (when w_q is given; over all 192 values)
//   c    = kv[:512] / sqrt(mean(kv[:512]^2) + eps) * w_kv     (when w_kv is given)
//   rope = pairs (a, b) of the last 64 values turned by the token's angles:
//          (a cos - b sin, b cos + a sin), pair k being values (2k, 2k + 1) or (k, k + 32)
// q' goes out as q_nope and q_pe, [c | rope(kv[512:])] to the token's cache row (bf16,
// or a 656-byte FP8 row).  Sums of squares and every product are fp32; each output
// value is rounded once, to bf16 (an FP8 row quantises the bf16-rounded latent, so that
// it holds the bytes that packing the bf16 row gives).
//
// Bound by memory: each value is read once and written once (4096 tokens x 128 heads,
// 413 MB: 60 us, the copy rate; with the head norm, whose instructions show, 68 to 70 us).  A
// warp takes eight heads of a token, or its cache row.
#include "mla_fp8.cuh"
#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kDQ = kDNope + kDRope;   // 192

struct AppendArgs {
  const __nv_bfloat16* q;
  int64_t q_token, q_head;          // strides, elements
  const __nv_bfloat16* kv;
  int64_t kv_token;
  const __nv_bfloat16* q_weight;    // [192] or null
  const __nv_bfloat16* kv_weight;   // [512] or null
  float eps;
  const float* cos_sin;             // [max_pos, 64]: cos | sin
  int max_pos;
  const int32_t* positions;
  const int32_t* slots;
  CacheView cv;
  unsigned char* rows_fp8;          // the FP8 pool, or null
  __nv_bfloat16* q_nope;
  __nv_bfloat16* q_pe;
  int* status;
  int N, H, units;                  // units (warps) per token: ceil(H / (4 kQuads)) + 1
};

__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The angles of rope chunk r (values 8 r .. 8 r + 7 of the 64): cs[e], sn[e] turn value e.
template <bool kInterleaved>
__device__ __forceinline__ void load_angles(const float* row, int r, float (&cs)[8], float (&sn)[8]) {
  if (kInterleaved) {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * r);
    const float4 s = *reinterpret_cast<const float4*>(row + 32 + 4 * r);
    cs[0] = cs[1] = c.x; cs[2] = cs[3] = c.y; cs[4] = cs[5] = c.z; cs[6] = cs[7] = c.w;
    sn[0] = sn[1] = s.x; sn[2] = sn[3] = s.y; sn[4] = sn[5] = s.z; sn[6] = sn[7] = s.w;
  } else {
    const float* base = row + 8 * (r & 3);
    const float4 c0 = *reinterpret_cast<const float4*>(base), c1 = *reinterpret_cast<const float4*>(base + 4);
    const float4 s0 = *reinterpret_cast<const float4*>(base + 32), s1 = *reinterpret_cast<const float4*>(base + 36);
    cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w; cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
    sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w; sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
  }
}
// Rope chunk r turned in place; the other half of a (k, k + 32) pair is four lanes away.
// Every lane of the warp takes part; `mine` lanes hold a rope chunk.
template <bool kInterleaved>
__device__ __forceinline__ void rotate8(float (&x)[8], const float (&cs)[8], const float (&sn)[8], int r, bool mine) {
  if (kInterleaved) {
    if (mine) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float a = x[k], b = x[k + 1];
        x[k] = a * cs[k] - b * sn[k];
        x[k + 1] = b * cs[k] + a * sn[k];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float other = __shfl_xor_sync(0xffffffffu, x[k], 4);
      if (mine) x[k] = r < 4 ? x[k] * cs[k] - other * sn[k] : x[k] * cs[k] + other * sn[k];
    }
  }
}

// The cache row of one token (a whole warp): lane l holds latent values
// [16 l, 16 l + 16), lanes 16..23 also rope chunk l - 16.
template <bool kInterleaved>
__device__ void append_row(const AppendArgs& a, int i, int pos, int lane) {
  const int slot = a.slots[i];
  if (slot < 0 || slot >= a.cv.num_blocks * kPage) {
    if (slot != -1 && lane == 0) atomicCAS(a.status, 0, MLA_ERR_DEVICE_CHECK);
    return;
  }
  const __nv_bfloat16* src = a.kv + (size_t)i * a.kv_token;
  const int r = lane - 16;
  const bool rope_lane = r >= 0 && r < 8;
  const uint4 u0 = *reinterpret_cast<const uint4*>(src + 16 * lane);
  const uint4 u1 = *reinterpret_cast<const uint4*>(src + 16 * lane + 8);
  const uint4 ur = rope_lane ? *reinterpret_cast<const uint4*>(src + kDLat + 8 * r) : make_uint4(0, 0, 0, 0);
  float x0[8], x1[8], xr[8], cs[8] = {}, sn[8] = {};
  unpack8(u0, x0);
  unpack8(u1, x1);
  unpack8(ur, xr);
  if (rope_lane) load_angles<kInterleaved>(a.cos_sin + (size_t)pos * kDRope, r, cs, sn);
  if (a.kv_weight) {
    float w0[8], w1[8], ss = 0.f;
    unpack8(*reinterpret_cast<const uint4*>(a.kv_weight + 16 * lane), w0);
    unpack8(*reinterpret_cast<const uint4*>(a.kv_weight + 16 * lane + 8), w1);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += x0[k] * x0[k] + x1[k] * x1[k];
    const float inv = rsqrtf(warp_sum(ss) * (1.f / kDLat) + a.eps);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x0[k] = x0[k] * inv * w0[k];
      x1[k] = x1[k] * inv * w1[k];
    }
  }
  rotate8<kInterleaved>(xr, cs, sn, r, rope_lane);
  const uint4 o0 = pack8(x0), o1 = pack8(x1), orr = pack8(xr);
  const int blk = slot / kPage, j = slot % kPage;
  if (a.rows_fp8) {
    float v0[8], v1[8], v[16], scale;
    unpack8(o0, v0);
    unpack8(o1, v1);
#pragma unroll
    for (int k = 0; k < 8; ++k) { v[k] = v0[k]; v[8 + k] = v1[k]; }
    const uint4 codes = fp8_quantise16(v, &scale);
    unsigned char* dst = a.rows_fp8 + (size_t)slot * kFp8RowBytes;
    *reinterpret_cast<uint4*>(dst + 16 * lane) = codes;
    if ((lane & 7) == 0) *reinterpret_cast<float*>(dst + kDLat + 4 * (lane >> 3)) = scale;
    if (rope_lane) *reinterpret_cast<uint4*>(dst + kDLat + 16 + 16 * r) = orr;
  } else {
    __nv_bfloat16* dst = const_cast<__nv_bfloat16*>(ckv_row_ptr(a.cv, blk, j)) + 16 * lane;
    *reinterpret_cast<uint4*>(dst) = o0;
    *reinterpret_cast<uint4*>(dst + 8) = o1;
    if (rope_lane)
      *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(kpe_row_ptr(a.cv, blk, j)) + 8 * r) = orr;
  }
}

// Sum over the 2 kHalf lanes that share lane / (2 kHalf).
template <int kHalf>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = kHalf; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float sum_squares(const float (&x)[8]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
  return s;
}

// Eight heads per warp: six loads in flight per lane.  Measured at 4096 tokens x 128 heads
// without norm: 4 heads 69.5 us, 8 heads 60.1 us (6.87 TB/s, the copy rate), 16 heads 60.4;
// 1 token 1.8, 1.8, 2.3 us.
constexpr int kQuads = 2;
// Blocks per SM, six (80 registers) or, with the norm and where all blocks are resident
// then, five (96): the norm's weights fit in registers, asked for with the rows.  With six
// they are read again for each four heads, from the L1.  287 tokens x 64 heads: 3.4 us with
// five, 3.9 with six; 4096 x 128: 74.6 and 70.3 us (with blocks of 256 threads, three of
// them per SM, 4.3 and 74.2; registers spilled for a launch's first rows cost as much as the
// rows).
constexpr int kBlocks = 6, kBlocksKeep = 5;

// Query rows of kQuads x 4 heads of a token by one warp.  Of four heads' 96 chunks a lane
// holds three: nope chunk lane % 16 of head lane / 16 and of head 2 + lane / 16, and rope
// chunk lane % 8 of head lane / 8, so that every lane works in every load, and the
// rotation runs once for four heads.
template <bool kInterleaved, bool kNorm, bool kKeep>
__global__ void __launch_bounds__(kAppendThreads, kKeep ? kBlocksKeep : kBlocks) rope_append_kernel(AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const long long token = unit / a.units;
  const int part = (int)(unit % a.units);
  if (token >= a.N) return;
  const int i = (int)token;
  const int pos = a.positions[i];
  const bool fine = pos >= 0 && pos < a.max_pos;
  if (part == a.units - 1) {
    if (fine) append_row<kInterleaved>(a, i, pos, lane);
    else if (lane == 0) atomicCAS(a.status, 0, MLA_ERR_DEVICE_CHECK);
    return;
  }
  const int h0 = part * 4 * kQuads;
  const int r = lane & 7;
  const __nv_bfloat16* src = a.q + (size_t)i * a.q_token;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 u[kQuads][3];
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int ha = h0 + 4 * k + (lane >> 4), hc = h0 + 4 * k + (lane >> 3);
    u[k][0] = ha < a.H ? *reinterpret_cast<const uint4*>(src + (size_t)ha * a.q_head + 8 * (lane & 15)) : zero;
    u[k][1] = ha + 2 < a.H ? *reinterpret_cast<const uint4*>(src + (size_t)(ha + 2) * a.q_head + 8 * (lane & 15)) : zero;
    u[k][2] = hc < a.H ? *reinterpret_cast<const uint4*>(src + (size_t)hc * a.q_head + kDNope + 8 * r) : zero;
  }
  // (the rows' loads are under way before the position, which the angles depend on, is here)
  if (!fine) return;
  float cs[8], sn[8];
  load_angles<kInterleaved>(a.cos_sin + (size_t)pos * kDRope, r, cs, sn);
  uint4 wn = zero, wr = zero;
  if (kKeep) {
    wn = *reinterpret_cast<const uint4*>(a.q_weight + 8 * (lane & 15));
    wr = *reinterpret_cast<const uint4*>(a.q_weight + kDNope + 8 * r);
  }
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int ha = h0 + 4 * k + (lane >> 4), hc = h0 + 4 * k + (lane >> 3);
    float xr[8];
    unpack8(u[k][2], xr);
    if (kNorm) {
      float xa[8], xb[8], w[8];
      unpack8(u[k][0], xa);
      unpack8(u[k][1], xb);
      const float sa = group_sum<8>(sum_squares(xa)), sb = group_sum<8>(sum_squares(xb));
      const float sr = group_sum<4>(sum_squares(xr));
      // the rope lanes of head h take its nope sum from lane 16 (h % 2) of a (h < 2) or b
      const int from = (lane & 8) << 1;
      const float fa = __shfl_sync(0xffffffffu, sa, from), fb = __shfl_sync(0xffffffffu, sb, from);
      const float inv = rsqrtf((sr + (lane < 16 ? fa : fb)) * (1.f / kDQ) + a.eps);
      const float ia = __shfl_sync(0xffffffffu, inv, (lane & 16) >> 1);
      const float ib = __shfl_sync(0xffffffffu, inv, 16 + ((lane & 16) >> 1));
      unpack8(kKeep ? wn : *reinterpret_cast<const uint4*>(a.q_weight + 8 * (lane & 15)), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xa[e] = xa[e] * ia * w[e];
        xb[e] = xb[e] * ib * w[e];
      }
      u[k][0] = pack8(xa);
      u[k][1] = pack8(xb);
      unpack8(kKeep ? wr : *reinterpret_cast<const uint4*>(a.q_weight + kDNope + 8 * r), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) xr[e] = xr[e] * inv * w[e];
    }
    rotate8<kInterleaved>(xr, cs, sn, r, true);
    __nv_bfloat16* nope = a.q_nope + ((size_t)i * a.H + ha) * kDNope + 8 * (lane & 15);
    if (ha < a.H) *reinterpret_cast<uint4*>(nope) = u[k][0];
    if (ha + 2 < a.H) *reinterpret_cast<uint4*>(nope + 2 * kDNope) = u[k][1];
    if (hc < a.H) *reinterpret_cast<uint4*>(a.q_pe + ((size_t)i * a.H + hc) * kDRope + 8 * r) = pack8(xr);
  }
}

}  // namespace

cudaError_t launch_rope_append(const AppendCall& c, cudaStream_t st) {
  AppendArgs a;
  a.q = c.q; a.q_token = c.q_token; a.q_head = c.q_head; a.kv = c.kv; a.kv_token = c.kv_token;
  a.q_weight = c.q_weight; a.kv_weight = c.kv_weight; a.eps = c.eps;
  a.cos_sin = c.cos_sin; a.max_pos = c.max_pos; a.positions = c.positions; a.slots = c.slots;
  a.cv = c.cv; a.rows_fp8 = c.rows_fp8; a.q_nope = c.q_nope; a.q_pe = c.q_pe;
  a.status = bmm_status_ptr();
  a.N = c.N; a.H = c.H;
  if (!a.status) return cudaErrorInvalidValue;
  a.units = (c.H + 4 * kQuads - 1) / (4 * kQuads) + 1;
  const long long ctas = ((long long)c.N * a.units + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  const dim3 grid((unsigned)ctas), block(kAppendThreads);
  if (c.q_weight && ctas <= (long long)kBlocksKeep * mla_device_sm_count())
    return c.interleaved ? launch_pdl(rope_append_kernel<true, true, true>, grid, block, 0, st, a)
                         : launch_pdl(rope_append_kernel<false, true, true>, grid, block, 0, st, a);
  if (c.q_weight)
    return c.interleaved ? launch_pdl(rope_append_kernel<true, true, false>, grid, block, 0, st, a)
                         : launch_pdl(rope_append_kernel<false, true, false>, grid, block, 0, st, a);
  return c.interleaved ? launch_pdl(rope_append_kernel<true, false, false>, grid, block, 0, st, a)
                       : launch_pdl(rope_append_kernel<false, false, false>, grid, block, 0, st, a);
}

}  // namespace mla
