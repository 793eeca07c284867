// Head RMSNorm and position rotation of q and k in one pass (between the QKV product and attention).
//
// For a head x of D elements in row r, with rstd = 1 / sqrt(mean(x^2) + eps) (1 without gamma), gamma
// (1 without) and the table row t(r) of cosines c and sines s, pair i < rot/2 is turned by its angle:
//
//   y = x * rstd * gamma,   out[a] = y[a] * c[i] - y[b] * s[i],   out[b] = y[b] * c[i] + y[a] * s[i]
//
// with (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved; elements from rot on are y.  Both forms
// are out[e] = rstd * (x[e] * A[e] + x[partner(e)] * B[e]) with A = gamma * c and B = -+ gamma[partner] * s,
// which depend on the row and the lane but not on the head: a warp makes them once (16 fp32 registers) and walks all
// the heads of its row with them, kRopeFlight steps in flight; with few rows the heads are shared by several warps.
//
// A head is D / 8 lanes of one 16-byte vector each (32 / 16 / 8 lanes for D = 256 / 128 / 64), so a warp
// step covers 1 / 2 / 4 heads; the sum of squares is a butterfly over the head's lanes.  The partner of
// the halves form is rot/16 lanes away and comes by four shuffles of packed bf16 pairs, that of the
// interleaved form is the other half of the same word.  A head is wholly in its warp's registers before
// any of it is written, so the output may be the input.
//
// Bound by HBM: 16896 rows of 36 heads of 256 take 105 us, 6.1 TB/s of reading and writing each element once (93% of a
// copy's rate); 4608 rows 31 us.  What it took: enough loads in flight per warp (one step at a time: 139 us) and few
// instructions per element (tables and gamma in registers for all heads of a row, fp32 in pairs).
#pragma once

#include "ptx.cuh"

namespace nvfp4 {

constexpr int kRopeFlight = 6;  // warp steps (of 256 / D heads) in flight together, a multiple of 3

struct RopeHeads {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  int64_t row, head, out_row, out_head;  // strides in elements
  const __nv_bfloat16* gamma;            // [D] or null
  int heads, chunks;                     // chunks of RopeArgs::steps warp steps
};

struct RopeArgs {
  RopeHeads q, k;
  int64_t rows;
  const float* cos;
  const float* sin;
  int64_t table_rows, ld_table;
  const int32_t* positions;  // [rows] or null
  int rot;
  int steps;  // warp steps per warp
  float eps;
};

// A packed bf16 pair as two fp32.
__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Both elements times 2^-70.
__device__ __forceinline__ uint32_t down70(uint32_t w) {
  const float2 x = bf16x2_to_float2(w);
  const __nv_bfloat162 b = __floats2bfloat162_rn(x.x * 0x1p-70f, x.y * 0x1p-70f);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// The sum of squares of a head from this lane's 8 elements of it, in each of the head's lanes.
template <int kLanes>
__device__ __forceinline__ float head_squares(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = bf16x2_to_float2(w[j]);
    s2 = fma2(x, x, s2);
  }
  float ss = s2.x + s2.y;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  return ss;
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int l = lane % kLanes;   // this lane's 8 elements of its head: [8 l, 8 l + 8)
  const uint32_t chunks = a.q.chunks + a.k.chunks;
  const uint32_t unit = blockIdx.x * 8u + (threadIdx.x >> 5);
  const uint32_t row = unit / chunks;
  if (row >= a.rows) return;  // warp-uniform
  int chunk = static_cast<int>(unit - row * chunks);
  const bool is_k = chunk >= a.q.chunks;
  const RopeHeads& h = is_k ? a.k : a.q;
  if (is_k) chunk -= a.q.chunks;
  int head = chunk * a.steps * kHeads + lane / kLanes;
  const int head_end = min(h.heads, (chunk + 1) * a.steps * kHeads);
  const __nv_bfloat16* xp = h.x + row * h.row + head * h.head + 8 * l;
  __nv_bfloat16* op = h.out + row * h.out_row + head * h.out_head + 8 * l;
  const int64_t x_step = kHeads * h.head, o_step = kHeads * h.out_head;

  uint4 v[kRopeFlight];
  auto load = [&] {
#pragma unroll
    for (int i = 0; i < kRopeFlight; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (head + i * kHeads < head_end) v[i] = *reinterpret_cast<const uint4*>(xp + i * x_step);
    }
  };
  load();

  // A and B of this lane's elements
  const int64_t pos = a.positions ? static_cast<int64_t>(a.positions[row])
                      : row < a.table_rows ? row : row % static_cast<uint32_t>(a.table_rows);
  const bool turned = 8 * l < a.rot && pos >= 0 && pos < a.table_rows;
  float A[8], Bm[8], gp[8];
  const int shift = a.rot / 16;  // lanes between the halves
  const bool second = 8 * l >= a.rot / 2;
  const int src = kInterleaved || !turned ? lane : (second ? lane - shift : lane + shift);
#pragma unroll
  for (int i = 0; i < 8; ++i) A[i] = gp[i] = 1.0f;
  if (h.gamma) {
    const uint4 g = __ldg(reinterpret_cast<const uint4*>(h.gamma + 8 * l));
    const uint4 p = __ldg(reinterpret_cast<const uint4*>(h.gamma + 8 * (l + src - lane)));
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      A[2 * i] = __uint_as_float(gw[i] << 16);
      A[2 * i + 1] = __uint_as_float(gw[i] & 0xFFFF0000u);
      gp[2 * i] = __uint_as_float(pw[i] << 16);
      gp[2 * i + 1] = __uint_as_float(pw[i] & 0xFFFF0000u);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) Bm[i] = 0.0f;
  if (turned) {
    if constexpr (kInterleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(a.cos + pos * a.ld_table + 4 * l));
      const float4 s = __ldg(reinterpret_cast<const float4*>(a.sin + pos * a.ld_table + 4 * l));
      const float cc[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g0 = A[2 * i], g1 = A[2 * i + 1];
        A[2 * i] = g0 * cc[i];
        Bm[2 * i] = -g1 * sv[i];
        A[2 * i + 1] = g1 * cc[i];
        Bm[2 * i + 1] = g0 * sv[i];
      }
    } else {
      const int64_t at = pos * a.ld_table + 8 * l - (second ? a.rot / 2 : 0);
      const float4 c0 = __ldg(reinterpret_cast<const float4*>(a.cos + at));
      const float4 c1 = __ldg(reinterpret_cast<const float4*>(a.cos + at + 4));
      const float4 s0 = __ldg(reinterpret_cast<const float4*>(a.sin + at));
      const float4 s1 = __ldg(reinterpret_cast<const float4*>(a.sin + at + 4));
      const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        A[i] *= cc[i];
        Bm[i] = (second ? gp[i] : -gp[i]) * sv[i];
      }
    }
  }

  // this lane's part of one head, from its 8 elements; every lane of the warp is here (partners' elements)
  auto turn = [&](uint4 u, float rstd) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t p;
      if constexpr (kInterleaved) {
        p = __byte_perm(w[j], 0u, 0x1032);
      } else {
        p = __shfl_sync(0xFFFFFFFFu, w[j], src);
      }
      p = turned ? p : 0u;  // an unturned element takes nothing, not even 0 * infinity, from another
      const float2 y = fma2(bf16x2_to_float2(p), make_float2(Bm[2 * j], Bm[2 * j + 1]),
                            mul2(bf16x2_to_float2(w[j]), make_float2(A[2 * j], A[2 * j + 1])));
      const float2 z = mul2(y, make_float2(rstd, rstd));
      const __nv_bfloat162 b = __floats2bfloat162_rn(z.x, z.y);
      r[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  };
  while (true) {
    // three steps at a time: their squares, one look whether they left fp32 (at all six 3% slower with pairs as neighbours,
    // at each step on its own 4 to 8%), their outputs
#pragma unroll
    for (int i0 = 0; i0 < kRopeFlight; i0 += 3) {
      float rstd[3], top = 0.0f;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        rstd[i] = 1.0f;
        if (h.gamma) {
          const float ss = head_squares<kLanes>(v[i0 + i]);
          top = fmaxf(top, ss);
          rstd[i] = rsqrtf(__fmaf_rn(ss, 1.0f / D, a.eps));
        }
      }
      if (__any_sync(0xFFFFFFFFu, top == INFINITY)) {
        // elements from about 1e18 on: the head is taken down by 2^70, beside which eps is nothing
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          uint4& u = v[i0 + i];
          const bool wide = rstd[i] == 0.0f;
          if (wide) u = make_uint4(down70(u.x), down70(u.y), down70(u.z), down70(u.w));
          const float ss = head_squares<kLanes>(u);
          if (wide) rstd[i] = rsqrtf(ss * (1.0f / D));
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint4 r = turn(v[i0 + i], rstd[i]);
        if (head + (i0 + i) * kHeads < head_end) *reinterpret_cast<uint4*>(op + (i0 + i) * o_step) = r;
      }
    }
    head += kRopeFlight * kHeads;
    if (head - lane / kLanes >= head_end) break;  // warp-uniform
    xp += kRopeFlight * x_step;
    op += kRopeFlight * o_step;
    load();
  }
}

}  // namespace nvfp4
