// Attention of a block's queries to an encoder's states of another length:
//
//   s = scale * q k^T over the sample's first kv_lens[b] keys,  p = exp(s - max s),  o = (p v) / sum p
//
// in one pass over the keys with a running maximum and sum: nothing of size queries x keys leaves the SM.
//
// A CTA has 128 query rows of one kv head (heads that share a kv head are packed into the rows: row
// tok * G + g for G heads per kv head), and walks the keys in tiles of 128.  S = Q K^T and O += P V run on
// tcgen05 with fp32 accumulators in TMEM: O in columns [0, D), two S tiles in [256, 512).  P replaces S in its
// own columns as bf16, from where it is the A operand of P V.  The MMA warp issues S of tile j + 1 before
// P V of tile j, so that the softmax of a tile runs while the tensor pipe does P V of the tile before and S of
// the tile after.
//
// Roles: warp 0 TMA producer; warp 1 MMA issuer (converged, one elected lane); warp 2 TMEM; warps 4-11
// softmax and output: two warpgroups, thread = one row, 64 of the tile's 128 columns each; the two
// threads of a row exchange their maxima through shared memory.
//
// Shared memory: Q, and a ring of 16 KB chunks that K and V share: a K chunk is 128 keys x 64 elements, a V chunk
// 64 * 128 / D keys x D elements, both in the 128-byte swizzle that TMA writes and the MMA reads (K as a
// K-major operand, V as an MN-major one).  A chunk is freed when its MMAs have completed.
//
// The reference maximum m is raised only when a row's new maximum exceeds it by more than 2^8 in the
// exponent's base-2 scale: then O and the sum are rescaled; otherwise p reaches at most 2^8, which changes no
// relative error.  p is rounded to bf16 for P V (2^-8 relative at most, independent from key to key, so about as large
// in the output as the rounding that follows); the sum is of the unrounded p in fp32.  (A second bf16 for what the
// rounding left out would make an infinity in V a NaN.)
//
// Keys past the length: their scores are set to -infinity, and their V rows in shared memory to zero (0 times an
// infinity or NaN behind a sample's last key would be NaN).  A sample without keys gives zeros and lse = -infinity.
//
// Few query rows (attention_kernel): the CTAs of a cluster take contiguous ranges of the key tiles and merge their (m, sum, O) through
// distributed shared memory in rank order.  A single token of 2 samples x 18 heads of 256 and 512 keys: 10.7 us (19 MB,
// 2.9 us of HBM time): launch, the first loads, one tile's chain of scores, softmax and product, and the merge, one after the
// other.
#pragma once

#include <cooperative_groups.h>

#include "gemm.cuh"

namespace nvfp4 {

// 2^x, 0 below the normals.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The exponent of p is s * score - ref with ref = s * m, m the row's reference maximum: one fma per score, s and ref
// made anew where m changes.  What the rounding of ref leaves out is common to the row's p and to their sum, and lies
// within the rounding of the fp32 scores.  From |ref| = 2^24 on it would be a factor of 2 and more between sums under
// two m, from 2^31 on p would leave fp32, and for the largest scales ref does.  There s is a power of two, which makes
// ref and the difference exact: the scale taken down to one, or less where |ref| would pass 2^101.  Scores that
// differ by 2^-16 of their value or more (single products) then have exponents 2^7 and more apart, as with the scale
// itself; what is nearer lies within the rounding of the fp32 sums.  (Subtracting m before the product is as exact: 2 x 2048
// queries, 1941 and 1500 keys, 24 heads of 64 took 76.7 us against 73.9; this 72.3 against 72.0.)
struct AttnExponent {
  float s, ref;
};

__device__ __forceinline__ AttnExponent attn_exponent(float m, float scale_log2) {
  AttnExponent x{scale_log2, m == -INFINITY ? 0.0f : m * scale_log2};
  if (!(fabsf(x.ref) < 16777216.0f)) {
    const int m_exp = (__float_as_int(m) >> 23) & 255, s_exp = __float_as_int(scale_log2) >> 23;
    x.s = __int_as_float(min(s_exp, 127 + 127 + 100 - m_exp) << 23);
    x.ref = m * x.s;
  }
  return x;
}

constexpr int kAttnMaxSplit = 8;  // CTAs of a cluster that share a query tile's keys

template <int D>
struct AttnCfg {
  static constexpr int BM = 128, BN = 128;
  static constexpr int THREADS = 384;
  static constexpr int CHUNK_BYTES = 16384;
  static constexpr int K_CHUNKS = D / 64;                 // chunks per tile, of K and of V
  static constexpr int V_CHUNKS = D / 64;
  static constexpr int V_KEYS = BN / V_CHUNKS;            // keys per V chunk
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int AUX_BYTES = 4096;
  static constexpr int STAGES = D == 256 ? 9 : 8;
  static constexpr int SMEM_BYTES = AUX_BYTES + 1023 + Q_BYTES + STAGES * CHUNK_BYTES;
  static constexpr int S_COL = 256;                       // TMEM column of the first S tile
  static constexpr int O_STRIDE = D + 4;                  // floats per row of the merge buffer
  static constexpr uint32_t IDESC_S = idesc_bf16(BM, BN, false);
  static constexpr uint32_t IDESC_O = idesc_bf16(BM, D, true);
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(Q_BYTES + STAGES * CHUNK_BYTES >= BM * O_STRIDE * 4, "the merge buffer reuses Q and the ring");
};

struct AttnArgs {
  int works, q_works, kv_heads;            // of the persistent kernel: pieces of work, those of one (kv head, sample)
  int q_len, kv_len, group, tok_per_tile;  // group: heads per kv head; tok_per_tile = 128 / group
  int qb_mul, kb_mul, kh_mul, vb_mul, vh_mul;  // 0 where q, k or v is broadcast over the batch or the heads
  const int32_t* kv_lens;
  float scale_log2;
  __nv_bfloat16* out;
  int64_t out_batch, out_row, out_head;
  float* lse;
  int heads;
  unsigned int* error_word;
  uint64_t timeout_ns;
#ifdef NVFP4_TEST_HOOKS
  int test_withhold;  // test builds only: the probabilities are never handed over, so the wait for them runs out
#endif
};

struct AttnMaps {
  CUtensorMap q, k, v;
};

template <int D>
__global__ void __launch_bounds__(384, 1)
    attention_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs args) {
  namespace cg = cooperative_groups;
  using C = AttnCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw);
  uint64_t* empty = full + C::STAGES;
  uint64_t* q_full = empty + C::STAGES;
  uint64_t* s_full = q_full + 1;   // [2]
  uint64_t* p_ready = s_full + 2;  // [2]
  uint64_t* o_done = p_ready + 2;
  uint64_t* drain = o_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_abort = abort_flag + 1;
  float* row_max = reinterpret_cast<float*>(smem_raw + 512);   // [2 tiles][2 halves][128]
  float* row_stat = reinterpret_cast<float*>(smem_raw + 2560); // [128]{m, sum} for the merge; first [128] of half sums
  uint8_t* qs = smem_raw + C::AUX_BYTES;
  qs += (1024u - (smem_u32(qs) & 1023u)) & 1023u;
  uint8_t* ring = qs + C::Q_BYTES;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const cg::cluster_group cluster = cg::this_cluster();
  const int S = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tok0 = static_cast<int>(blockIdx.x / S) * args.tok_per_tile;
  const int kvh = blockIdx.y, b = blockIdx.z;
  int len = args.kv_len;
  if (args.kv_lens != nullptr) len = max(0, min(len, args.kv_lens[b]));
  const int tiles_all = (len + C::BN - 1) / C::BN;
  const int per = (tiles_all + S - 1) / S;
  const int t0 = min(tiles_all, rank * per), t1 = min(tiles_all, t0 + per);
  const int T = t1 - t0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 8);
    }
    mbar_init(o_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  float m = -INFINITY, sum = 0.0f;  // softmax threads: this row's reference maximum and (half) sum
  bool ok = true;

  if (warp == 0) {
    if (lane == 0 && T > 0) {
      // ------------------------------------------------------------------ TMA producer
      const int rows = args.tok_per_tile * args.group;
      mbar_arrive_expect_tx(q_full, rows * D * 2);
      for (int s = 0; s < D / 64; ++s)
        tma_load_4d(qs + s * (C::BM * 128), &maps.q, q_full, s * 64, kvh * args.group, tok0, b * args.qb_mul);
      int n = 0;  // chunks issued
      auto slot = [&]() -> uint8_t* {
        const int st = n % C::STAGES;
        if (!mbar_wait(&empty[st], ((n / C::STAGES) & 1) ^ 1, abort_flag, args.timeout_ns)) return nullptr;
        mbar_arrive_expect_tx(&full[st], C::CHUNK_BYTES);
        return ring + st * C::CHUNK_BYTES;
      };
      auto load_k = [&](int t) {
        for (int c = 0; c < C::K_CHUNKS; ++c) {
          uint8_t* dst = slot();
          if (dst == nullptr) return false;
          tma_load_4d(dst, &maps.k, &full[n % C::STAGES], c * 64, kvh * args.kh_mul, t * C::BN, b * args.kb_mul);
          ++n;
        }
        return true;
      };
      ok = load_k(t0);
      for (int t = t0; ok && t < t1; ++t) {
        if (t + 1 < t1) ok = load_k(t + 1);
        for (int c = 0; ok && c < C::V_CHUNKS; ++c) {
          uint8_t* dst = slot();
          if (dst == nullptr) {
            ok = false;
            break;
          }
          for (int s = 0; s < D / 64; ++s)
            tma_load_4d(dst + s * (C::V_KEYS * 128), &maps.v, &full[n % C::STAGES], s * 64, kvh * args.vh_mul,
                        t * C::BN + c * C::V_KEYS, b * args.vb_mul);
          ++n;
        }
      }
      if (!ok) raise_device_error(args.error_word, kErrTimeout, abort_flag);
      // The copies in flight write this CTA's shared memory: wait for them before it ends.  Whatever became of the others:
      // the MMA warp, which waits for the same copies, may have given up.
      bool landed = mbar_wait(q_full, 0, never_abort, args.timeout_ns);
      for (int i = max(0, n - C::STAGES); landed && i < n; ++i)
        landed = mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, never_abort, args.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (T > 0) {
      // ------------------------------------------------------------------ MMA issuer
      const uint32_t t_base = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
      const uint64_t q_desc = desc_kmajor_swizzled<128>(smem_u32(qs));
      const uint64_t k_desc = desc_kmajor_swizzled<128>(smem_u32(ring));
      const uint64_t v_desc = desc_mnmajor_sw128(smem_u32(ring), C::V_KEYS * 128);
      int st = 0;
      uint32_t phase = 0;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, args.timeout_ns));
        tc_fence_after();
        return got;
      };
      auto advance = [&] {
        tc_commit_warp(&empty[st]);
        if (++st == C::STAGES) {
          st = 0;
          phase ^= 1u;
        }
      };
      auto issue_s = [&](int j) {
#pragma unroll
        for (int c = 0; c < C::K_CHUNKS; ++c) {
          if (!wait(&full[st], phase)) return false;
          const uint64_t kd = k_desc + st * (C::CHUNK_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_bf16_ss_warp(t_base + C::S_COL + (j & 1) * C::BN, q_desc + c * (C::BM * 128 >> 4) + 2 * k, kd + 2 * k,
                                C::IDESC_S, c | k);
          advance();
        }
        tc_commit_warp(&s_full[j & 1]);
        return true;
      };
      ok = wait(q_full, 0) && issue_s(0);
      for (int j = 0; ok && j < T; ++j) {
        if (j + 1 < T) ok = issue_s(j + 1);
        if (!ok || !(ok = wait(&p_ready[j & 1], (j >> 1) & 1))) break;
        for (int c = 0; c < C::V_CHUNKS; ++c) {
          if (!(ok = wait(&full[st], phase))) break;
          const uint64_t vd = v_desc + st * (C::CHUNK_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < C::V_KEYS / 16; ++k)
            tc_mma_bf16_ts_warp(t_base, t_base + C::S_COL + (j & 1) * C::BN + c * (C::V_KEYS / 2) + k * 8,
                                vd + k * (16 * 128 >> 4), C::IDESC_O, j | c | k);
          advance();
        }
        if (ok) tc_commit_warp(o_done);
      }
      if (!ok && lane == 0) raise_device_error(args.error_word, kErrTimeout, abort_flag);
      tc_commit_warp(drain);
      mbar_wait(drain, 0, never_abort, args.timeout_ns);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // -------------------------------------------------------------------- softmax
    const int h = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    // 32 rows without a query (a single token has one row): their P stays as it is, and so do only their outputs
    const bool idle = quad * 32 >= min(args.tok_per_tile, args.q_len - tok0) * args.group;
    AttnExponent x{};
    for (int j = 0; j < T; ++j) {
      const uint32_t t_s = t_lane + C::S_COL + (j & 1) * C::BN;
      // a warp whose wait ran out goes on through the barriers of its pair, so that none waits there for good
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[j & 1], (j >> 1) & 1, abort_flag, args.timeout_ns));
      tc_fence_after();
      if (!idle) {
        uint32_t raw[2][32];
        tmem_ld_32x32b_x32(t_s + h * 64, raw[0]);
        tmem_ld_32x32b_x32(t_s + h * 64 + 32, raw[1]);
        tmem_ld_wait();
        const int left = len - (t0 + j) * C::BN - h * 64;  // keys of this half
        if (left < 64) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= left) raw[i >> 5][i & 31] = 0xFF800000u;  // -infinity
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 64; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], __uint_as_float(raw[i >> 5][i & 31]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        float* mine = row_max + (j & 1) * 256;
        mine[h * 128 + row] = mx;
        named_barrier_sync(1 + quad, 64);  // the two warps of these 32 rows; also: both have read their half of S
        if (!ok) continue;
        mx = fmaxf(mx, mine[(h ^ 1) * 128 + row]);
        if (j == 0) {
          m = mx;
          x = attn_exponent(m, args.scale_log2);
        } else {
          const bool grow = (mx - m) * args.scale_log2 > 8.0f;
          if (__any_sync(0xFFFFFFFFu, grow)) {
            // the rows that need it; a neighbour's bits do not depend on them
            const float f = grow ? ex2((m - mx) * args.scale_log2) : 1.0f;
            if (grow) {
              m = mx;
              x = attn_exponent(m, args.scale_log2);
            }
            sum *= f;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_done, (j - 1) & 1, abort_flag, args.timeout_ns));
            if (!ok) continue;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(t_lane + h * (D / 2) + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st_32x32b_x32(t_lane + h * (D / 2) + c, o);
            }
            tmem_st_wait();
          }
        }
        float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const float a = ex2(__fmaf_rn(__uint_as_float(raw[i >> 5][i & 31]), x.s, -x.ref));
          const float c = ex2(__fmaf_rn(__uint_as_float(raw[i >> 5][(i & 31) + 1]), x.s, -x.ref));
          s4[i & 2] += a;
          s4[(i & 2) + 1] += c;
          const __nv_bfloat162 v = __floats2bfloat162_rn(a, c);
          p[i >> 1] = *reinterpret_cast<const uint32_t*>(&v);
        }
        sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        tmem_st_32x32b_x32(t_s + h * 32, p);
      }
      // the last tile's V rows behind the sample's last key
      const int v_first = (j + 1 < T ? 2 : 1) * C::K_CHUNKS + j * (C::K_CHUNKS + C::V_CHUNKS);  // its first chunk
      const int keys = len - (t0 + j) * C::BN;
      if (keys < C::BN && len < args.kv_len) {
        for (int c = keys / C::V_KEYS; c < C::V_CHUNKS; ++c) {
          const int n = v_first + c;
          if (!__all_sync(0xFFFFFFFFu,
                          mbar_wait(&full[n % C::STAGES], (n / C::STAGES) & 1, abort_flag, args.timeout_ns))) {
            ok = false;
            break;
          }
          uint8_t* chunk = ring + (n % C::STAGES) * C::CHUNK_BYTES;
          const int from = max(0, keys - c * C::V_KEYS) * 128;  // whole rows: the swizzle stays within a row
          for (int s = 0; s < D / 64; ++s)
            for (int at = from + (threadIdx.x - 128) * 16; at < C::V_KEYS * 128; at += 256 * 16)
              *reinterpret_cast<uint4*>(chunk + s * (C::V_KEYS * 128) + at) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        if (!ok) continue;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
#ifdef NVFP4_TEST_HOOKS
      if (args.test_withhold) continue;
#endif
      if (lane == 0) mbar_arrive(&p_ready[j & 1]);
    }
    // P V of the last tile but one may still run (its S was issued before it), and a wait for a parity tells the last
    // phase from the one two before only once the one between has passed
    if (ok && T > 1) ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_done, (T - 2) & 1, abort_flag, args.timeout_ns));
    if (ok && T > 0) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_done, (T - 1) & 1, abort_flag, args.timeout_ns));
      tc_fence_after();
    }
    if (!ok && lane == 0) raise_device_error(args.error_word, kErrTimeout, abort_flag);
    // the row's sum is that of its two halves
    row_max[h * 128 + row] = sum;
    named_barrier_sync(1 + quad, 64);
    sum += row_max[(h ^ 1) * 128 + row];
    if (h == 0) {
      row_stat[2 * row] = m;
      row_stat[2 * row + 1] = sum;
    }
  }

  // ---------------------------------------------------------------------- output
  if (S > 1) cluster_sync();
  const int rows = args.tok_per_tile * args.group;
  const int toks = min(args.tok_per_tile, args.q_len - tok0);
  if (warp >= 4) {
    const int h = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const int tok = row / args.group, g = row % args.group;
    const bool live = row < rows && tok < toks && ok;
    float top = m, total = sum;
    if (S > 1 && live) {
      float2 st[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        st[r] = r < S ? *reinterpret_cast<const float2*>(cluster.map_shared_rank(row_stat, r) + 2 * row)
                      : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int r = 0; r < 8; ++r) top = fmaxf(top, st[r].x);
      total = 0.0f;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (st[r].x > -INFINITY || !(st[r].y == 0.0f))
          total += st[r].y * (st[r].x == top ? 1.0f : ex2((st[r].x - top) * args.scale_log2));
    }
    float f = total == 0.0f ? 0.0f : __fdividef(1.0f, total);
    if (S > 1 && m != top) f *= ex2((m - top) * args.scale_log2);
    const int64_t head = static_cast<int64_t>(kvh) * args.group + g;
    if (live && args.lse != nullptr && h == 0 && rank == 0)
      args.lse[(b * static_cast<int64_t>(args.heads) + head) * args.q_len + tok0 + tok] =
          total == 0.0f ? -INFINITY : __fmaf_rn(top, args.scale_log2, log2f(total)) * 0.6931471805599453f;
    __nv_bfloat16* out = args.out + b * args.out_batch + (tok0 + static_cast<int64_t>(tok)) * args.out_row + head * args.out_head;
    float* part = reinterpret_cast<float*>(qs) + row * C::O_STRIDE;
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
      if (!__any_sync(0xFFFFFFFFu, live)) break;
      const int col = h * (D / 2) + c;
      uint32_t o[32];
      if (T > 0) {
        tmem_ld_32x32b_x32(t_lane + col, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0u;
      }
      if (S > 1) {
        if (live)
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(part + col + i) =
                make_float4(__uint_as_float(o[i]) * f, __uint_as_float(o[i + 1]) * f, __uint_as_float(o[i + 2]) * f,
                            __uint_as_float(o[i + 3]) * f);
      } else if (live) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[i + 2 * k]) * f, __uint_as_float(o[i + 2 * k + 1]) * f);
            w[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          *reinterpret_cast<uint4*>(out + col + i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  __syncwarp();
  if (S > 1) {
    cluster_sync();
    // every CTA adds a share of the rows' partial outputs, in rank order
    const int n4 = toks * args.group * (D / 4);
    for (int idx = static_cast<int>(threadIdx.x) * S + rank; idx < n4; idx += S * C::THREADS) {
      const int row = idx / (D / 4), col = (idx % (D / 4)) * 4;
      float4 p[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        p[r] = r < S ? *reinterpret_cast<const float4*>(cluster.map_shared_rank(reinterpret_cast<float*>(qs), r) +
                                                        row * C::O_STRIDE + col)
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float4 a = p[0];
#pragma unroll
      for (int r = 1; r < 8; ++r) {
        a.x += p[r].x;
        a.y += p[r].y;
        a.z += p[r].z;
        a.w += p[r].w;
      }
      const int tok = row / args.group, g = row % args.group;
      __nv_bfloat16* out = args.out + b * args.out_batch + (tok0 + static_cast<int64_t>(tok)) * args.out_row +
                           (static_cast<int64_t>(kvh) * args.group + g) * args.out_head + col;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
      *reinterpret_cast<uint2*>(out) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its shared memory is read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ------------------------------------------------------------------------------------------
// Many query rows: a persistent kernel, one CTA per SM, over (query rows, kv head, sample)
// ------------------------------------------------------------------------------------------
//
// As above, without the key split, and with what follows one piece of work overlapping the next: the ring runs on
// into the next piece's keys, its queries are loaded as soon as the last S product has read the current ones, and its
// first scores are computed while the outputs of the current one leave TMEM.  For head_dim 64 and 128 the pieces of a round go to
// the CTAs forwards and backwards in turn, so that samples of different lengths even out (2 x 2048 queries, 1941 and 1500
// keys, 24 heads of 64: 71.8 us, all rounds forwards 76.9; the pairs of 256 lost 2% of 4096 x 512 by it).
//
// head_dim 64 and 128 (256: below): the exponentials take as long as the tensor work or longer, so two tiles of 128 rows share each key
// tile, one per softmax warpgroup (a thread has a whole row, no exchange): while one waits for its products the
// other has the exponential units.  The order on the tensor pipe is  P0 V, S0 of the next tile, P1 V, S1 of the next
// tile;  a chunk of K or V is freed after its second use.  head_dim 64, whose exponentials take four times its tensor
// work, keeps P in columns of its own and computes S of the next tile as soon as a warpgroup has read S.  The two
// warpgroups take turns with their exponentials: left alone they fall into step, both idle while the other waits
// (the same case, all forwards: 95 us, in turns 77 us; moving two or three eighths of the exponentials to a
// polynomial on the fp32 pipe gained 6% without the turns and lost 5 to 14% with them).
//
// Outputs: a warpgroup packs its rows to bf16 in registers, frees O, and writes them through a small piece of shared
// memory, so that four lanes write 64 consecutive bytes of a row (a lane writing its own row, 16 bytes per
// instruction, took 8400 cycles per tile of 128 x 256, as much as the products of four key tiles).
template <int D>
struct AttnRowsCfg {
  static constexpr int NQ = 2;                            // query tiles
  static constexpr int BM = 128, BN = 128;
  static constexpr int THREADS = 384;
  static constexpr int CHUNK_BYTES = 16384;
  static constexpr int CHUNKS = D / 64;                   // per key tile, of K and of V
  static constexpr int V_KEYS = BN / CHUNKS;
  static constexpr int Q_TILE = BM * D * 2;
  static constexpr int Q_BYTES = NQ * Q_TILE;
  static constexpr int AUX_BYTES = 1024;
  static constexpr int OUT_PITCH = 80;                    // per softmax warp: 32 rows x 64 bytes of output
  static constexpr int OUT_BYTES = 8 * 32 * OUT_PITCH;
  static constexpr int FIT = (232448 - AUX_BYTES - 1023 - Q_BYTES - OUT_BYTES) / CHUNK_BYTES;
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int SMEM_BYTES = AUX_BYTES + 1023 + Q_BYTES + STAGES * CHUNK_BYTES + OUT_BYTES;
  static constexpr int S_COL = 256;                       // TMEM column of the first S tile
  // head_dim 64 leaves TMEM columns for P of its own, so that the next scores need not wait for P V
  static constexpr bool OWN_P = D == 64;
  static constexpr bool K_FIRST = OWN_P;                  // S of the next tile is issued before P V of this one
  static constexpr int P_COL = OWN_P ? 128 : S_COL;       // of P tile 0
  static constexpr int P_STRIDE = OWN_P ? 64 : BN;
  static constexpr int P_ARRIVALS = 4;                    // warps that write a P tile
  static constexpr uint32_t IDESC_S = idesc_bf16(BM, BN, false);
  static constexpr uint32_t IDESC_O = idesc_bf16(BM, D, true);
  // V of a tile and K of the next one fit at once (both are held until their second use), so the
  // slot of a V chunk that a softmax warp waits for was last used by an earlier tile's V or by K up to its own
  static_assert(STAGES >= 2 * CHUNKS, "ring");
};

// A piece of work: query tokens from tok0, kv head, sample, and its key tiles.
struct AttnWork {
  int tok0, kvh, b, len, tiles;
};

template <int NQ>
__device__ __forceinline__ AttnWork attn_work(const AttnArgs& a, int i) {
  AttnWork w;
  const int q = i % a.q_works;
  i /= a.q_works;
  w.kvh = i % a.kv_heads;
  w.b = i / a.kv_heads;
  w.tok0 = q * NQ * a.tok_per_tile;
  w.len = a.kv_len;
  if (a.kv_lens != nullptr) w.len = max(0, min(w.len, __ldg(a.kv_lens + w.b)));
  w.tiles = (w.len + 127) / 128;
  return w;
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    attention_rows_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs args) {
  using C = AttnRowsCfg<D>;
  constexpr int NQ = C::NQ;
  extern __shared__ uint8_t smem_raw[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw);
  uint64_t* empty = full + C::STAGES;
  uint64_t* q_full = empty + C::STAGES;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;   // [2]
  uint64_t* p_ready = s_full + 2;   // [2]
  uint64_t* o_done = p_ready + 2;   // [2]
  uint64_t* o_free = o_done + 2;    // [2]
  uint64_t* s_free = o_free + 2;    // [2]: OWN_P
  uint64_t* drain = s_free + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_abort = abort_flag + 1;
  uint8_t* qs = smem_raw + C::AUX_BYTES;
  qs += (1024u - (smem_u32(qs) & 1023u)) & 1023u;
  uint8_t* ring = qs + C::Q_BYTES;
  uint8_t* stage_out = ring + C::STAGES * C::CHUNK_BYTES;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], C::P_ARRIVALS);
      mbar_init(&o_done[i], 1);
      mbar_init(&o_free[i], C::P_ARRIVALS);
      mbar_init(&s_free[i], C::P_ARRIVALS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  bool ok = true;

  if (warp < 4) {
    regs_decrease<56>();
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------------- TMA producer
        int n = 0, w = 0;  // chunks issued, pieces of work with keys
        auto load = [&](const CUtensorMap* map, int boxes, int x_step, int y, int row, int z, int box_bytes) {
          const int st = n % C::STAGES;
          if (!mbar_wait(&empty[st], ((n / C::STAGES) & 1) ^ 1, abort_flag, args.timeout_ns)) return false;
          mbar_arrive_expect_tx(&full[st], C::CHUNK_BYTES);
          for (int s = 0; s < boxes; ++s)
            tma_load_4d(ring + st * C::CHUNK_BYTES + s * box_bytes, map, &full[st], x_step + s * 64, y, row, z);
          ++n;
          return true;
        };
        for (int i = blockIdx.x, step = 2 * (gridDim.x - blockIdx.x) - 1; ok && i < args.works; i += step, step = 2 * gridDim.x - step) {
          const AttnWork wk = attn_work<NQ>(args, i);
          if (wk.tiles == 0) continue;
          auto load_k = [&](int t) {
            for (int c = 0; ok && c < C::CHUNKS; ++c)
              ok = load(&maps.k, 1, c * 64, wk.kvh * args.kh_mul, t * C::BN, wk.b * args.kb_mul, 0);
          };
          auto load_v = [&](int t) {
            for (int c = 0; ok && c < C::CHUNKS; ++c)
              ok = load(&maps.v, C::CHUNKS, 0, wk.kvh * args.vh_mul, t * C::BN + c * C::V_KEYS, wk.b * args.vb_mul,
                        C::V_KEYS * 128);
          };
          // the first keys do not wait for the queries' buffer
          load_k(0);
          if (ok) ok = mbar_wait(q_empty, (w & 1) ^ 1, abort_flag, args.timeout_ns);
          if (!ok) break;
          mbar_arrive_expect_tx(q_full, NQ * args.tok_per_tile * args.group * D * 2);
          for (int q = 0; q < NQ; ++q)
            for (int s = 0; s < C::CHUNKS; ++s)
              tma_load_4d(qs + q * C::Q_TILE + s * (C::BM * 128), &maps.q, q_full, s * 64, wk.kvh * args.group,
                          wk.tok0 + q * args.tok_per_tile, wk.b * args.qb_mul);
          ++w;
          for (int t = 0; ok && t < wk.tiles; ++t) {
            // the order of use
            if (C::K_FIRST && t + 1 < wk.tiles) load_k(t + 1);
            load_v(t);
            if (!C::K_FIRST && t + 1 < wk.tiles) load_k(t + 1);
          }
        }
        if (!ok) raise_device_error(args.error_word, kErrTimeout, abort_flag);
        // the copies in flight, as above
        bool landed = w == 0 || mbar_wait(q_full, (w - 1) & 1, never_abort, args.timeout_ns);
        for (int i = max(0, n - C::STAGES); landed && i < n; ++i)
          landed = mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, never_abort, args.timeout_ns);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------------ MMA issuer
      const uint32_t t_base = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
      const uint64_t q_desc = desc_kmajor_swizzled<128>(smem_u32(qs));
      const uint64_t k_desc = desc_kmajor_swizzled<128>(smem_u32(ring));
      const uint64_t v_desc = desc_mnmajor_sw128(smem_u32(ring), C::V_KEYS * 128);
      int st = 0, n = 0, w = 0;  // ring position; key tiles and pieces of work done
      uint32_t phase = 0;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, args.timeout_ns));
        tc_fence_after();
        return got;
      };
      // chunks at ring position `at`; `first`: wait for each, `last`: free each
      auto issue_s = [&](int q, int buf, int at, uint32_t ph, bool first, bool last) {
#pragma unroll
        for (int c = 0; c < C::CHUNKS; ++c) {
          if (first && !wait(&full[at], ph)) return false;
          const uint64_t kd = k_desc + at * (C::CHUNK_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_bf16_ss_warp(t_base + C::S_COL + buf * C::BN, q_desc + ((q * C::Q_TILE + c * (C::BM * 128)) >> 4) + 2 * k,
                                kd + 2 * k, C::IDESC_S, c | k);
          if (last) tc_commit_warp(&empty[at]);
          if (++at == C::STAGES) {
            at = 0;
            ph ^= 1u;
          }
        }
        tc_commit_warp(&s_full[buf]);
        return true;
      };
      auto issue_o = [&](int q, int buf, int at, uint32_t ph, bool first, bool last, int accumulate) {
#pragma unroll
        for (int c = 0; c < C::CHUNKS; ++c) {
          if (first && !wait(&full[at], ph)) return false;
          const uint64_t vd = v_desc + at * (C::CHUNK_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < C::V_KEYS / 16; ++k)
            tc_mma_bf16_ts_warp(t_base + q * D, t_base + C::P_COL + buf * C::P_STRIDE + c * (C::V_KEYS / 2) + k * 8,
                                vd + k * (16 * 128 >> 4), C::IDESC_O, accumulate | c | k);
          if (last) tc_commit_warp(&empty[at]);
          if (++at == C::STAGES) {
            at = 0;
            ph ^= 1u;
          }
        }
        tc_commit_warp(&o_done[q]);
        return true;
      };
      auto skip = [&](int chunks) {
        st += chunks;
        if (st >= C::STAGES) {
          st -= C::STAGES;
          phase ^= 1u;
        }
      };
      for (int i = blockIdx.x, step = 2 * (gridDim.x - blockIdx.x) - 1; ok && i < args.works; i += step, step = 2 * gridDim.x - step) {
        const AttnWork wk = attn_work<NQ>(args, i);
        if (wk.tiles == 0) continue;
        if (!(ok = wait(q_full, w & 1))) break;
        ok = issue_s(0, 0, st, phase, true, false) && issue_s(1, 1, st, phase, false, true);
        skip(C::CHUNKS);
        if (wk.tiles == 1) tc_commit_warp(q_empty);
        for (int j = 0; ok && j < wk.tiles; ++j, ++n) {
          const bool more = j + 1 < wk.tiles;
          if (C::OWN_P && more) {
            // the next scores as soon as these have been read
            for (int q = 0; ok && q < 2; ++q)
              ok = wait(&s_free[q], n & 1) && issue_s(q, q, st, phase, q == 0, q == 1);
            skip(C::CHUNKS);
          }
          const int v_st = st;
          const uint32_t v_ph = phase;
          skip(C::CHUNKS);
          for (int q = 0; ok && q < 2; ++q) {
            if (j == 0) ok = wait(&o_free[q], (w & 1) ^ 1);
            ok = ok && wait(&p_ready[q], n & 1) && issue_o(q, q, v_st, v_ph, q == 0, q == 1, j);
            if (!C::OWN_P && more) ok = ok && issue_s(q, q, st, phase, q == 0, q == 1);
          }
          if (!C::OWN_P && more) skip(C::CHUNKS);
          if (j + 2 == wk.tiles) tc_commit_warp(q_empty);
        }
        ++w;
      }
      if (!ok && lane == 0) raise_device_error(args.error_word, kErrTimeout, abort_flag);
      tc_commit_warp(drain);
      mbar_wait(drain, 0, never_abort, args.timeout_ns);
      __syncwarp();
    }
  } else {
    regs_increase<224>();
    // -------------------------------------------------------------------- softmax and output
    constexpr int COLS = C::BN, O_COLS = D;   // of a key tile and of O, per thread
    const int q = (warp - 4) >> 2, quad = warp & 3;  // query tile of this warpgroup
    const int row = quad * 32 + lane;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t t_o = t_lane + q * D;
    const int tok_in = row / args.group, g = row % args.group;
    int n = 0, chunk0 = 0;  // key tiles done; ring chunks of the work before
    if (q == 1) named_barrier_arrive(1, 256);  // warpgroup 0 begins
    for (int i = blockIdx.x, step = 2 * (gridDim.x - blockIdx.x) - 1; i < args.works; i += step, step = 2 * gridDim.x - step) {
      const AttnWork wk = attn_work<NQ>(args, i);
      const int T = wk.tiles;
      float m = -INFINITY, sum = 0.0f;
      AttnExponent x{};
      for (int j = 0; j < T; ++j, ++n) {
        const uint32_t t_s = t_lane + C::S_COL + q * C::BN;
        // a warp whose wait ran out goes on through the turns, so that the other warpgroup does not wait there for good
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[q], n & 1, abort_flag, args.timeout_ns));
        tc_fence_after();
        uint32_t raw[COLS];
#pragma unroll
        for (int c = 0; c < COLS; c += 32)
          tmem_ld_32x32b_x32(t_s + c, *reinterpret_cast<uint32_t(*)[32]>(raw + c));
        tmem_ld_wait();
        if constexpr (C::OWN_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[q]);
        }
        const int left = wk.len - j * C::BN;  // keys of this tile
        if (left < COLS) {
#pragma unroll
          for (int k = 0; k < COLS; ++k)
            if (k >= left) raw[k] = 0xFF800000u;  // -infinity
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < COLS; k += 2)
          mx4[(k >> 1) & 3] = fmaxf(fmaxf(mx4[(k >> 1) & 3], __uint_as_float(raw[k])), __uint_as_float(raw[k + 1]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        if (j == 0) {
          m = mx;
          x = attn_exponent(m, args.scale_log2);
        } else {
          const bool grow = (mx - m) * args.scale_log2 > 8.0f;
          if (__any_sync(0xFFFFFFFFu, grow)) {
            // the rows that need it; a neighbour's bits do not depend on them
            const float f = grow ? ex2((m - mx) * args.scale_log2) : 1.0f;
            if (grow) {
              m = mx;
              x = attn_exponent(m, args.scale_log2);
            }
            sum *= f;
            if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&o_done[q], (n - 1) & 1, abort_flag, args.timeout_ns));
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < O_COLS; c += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(t_o + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st_32x32b_x32(t_o + c, o);
            }
            tmem_st_wait();
          }
        }
        if (C::OWN_P && j > 0) {
          // P V of the tile before has read P
          if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&o_done[q], (n - 1) & 1, abort_flag, args.timeout_ns));
          tc_fence_after();
        }
        named_barrier_sync(1 + q, 256);  // this warpgroup's turn
        const uint32_t t_p = t_lane + C::P_COL + q * C::P_STRIDE;
        const float2 scale2 = make_float2(x.s, x.s), ref2 = make_float2(-x.ref, -x.ref);
        float2 s2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float2 e = fma2(make_float2(__uint_as_float(raw[c + k]), __uint_as_float(raw[c + k + 1])), scale2, ref2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            s2[(k >> 1) & 1] = add2(s2[(k >> 1) & 1], e);
            const __nv_bfloat162 v = __floats2bfloat162_rn(e.x, e.y);
            p[k >> 1] = *reinterpret_cast<const uint32_t*>(&v);
          }
          tmem_st_32x32b_x16(t_p + c / 2, p);
        }
        named_barrier_arrive(2 - q, 256);  // the other's turn (earlier, they overlap and fall into step)
        if (!ok) continue;
        sum += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
        // the last tile's V rows behind the sample's last key (both query tiles' warps do it: the same zeros)
        const int keys = wk.len - j * C::BN;
        if (keys < C::BN && wk.len < args.kv_len) {
          // chunks of this work before V of tile j
          const int before = C::K_FIRST ? (min(j + 2, T) + j) * C::CHUNKS : (2 * j + 1) * C::CHUNKS;
          for (int c = keys / C::V_KEYS; c < C::CHUNKS; ++c) {
            const int at = chunk0 + before + c;
            if (ok)
              ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[at % C::STAGES], (at / C::STAGES) & 1, abort_flag, args.timeout_ns));
            if (!ok) break;
            uint8_t* chunk = ring + (at % C::STAGES) * C::CHUNK_BYTES;
            const int from = max(0, keys - c * C::V_KEYS) * 128;  // whole rows: the swizzle stays within a row
            for (int s = 0; s < C::CHUNKS; ++s)
              for (int b = from + row * 16; b < C::V_KEYS * 128; b += 128 * 16)
                *reinterpret_cast<uint4*>(chunk + s * (C::V_KEYS * 128) + b) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          if (!ok) continue;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
#ifdef NVFP4_TEST_HOOKS
        if (args.test_withhold) continue;
#endif
        if (lane == 0) mbar_arrive(&p_ready[q]);
      }
      chunk0 += 2 * T * C::CHUNKS;
      // (the phase before the last has passed: it was waited for, or lies before S of the last tile)
      if (ok && T > 0) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&o_done[q], (n - 1) & 1, abort_flag, args.timeout_ns));
        tc_fence_after();
      }
      if (!ok && lane == 0) raise_device_error(args.error_word, kErrTimeout, abort_flag);
      const int tok = wk.tok0 + q * args.tok_per_tile + tok_in;
      const bool live = ok && tok_in < args.tok_per_tile && tok < args.q_len;
      const float f = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
      if (live && args.lse != nullptr)
        args.lse[(wk.b * static_cast<int64_t>(args.heads) + wk.kvh * args.group + g) * args.q_len + tok] =
            sum == 0.0f ? -INFINITY : __fmaf_rn(m, args.scale_log2, log2f(sum)) * 0.6931471805599453f;
      // the row's outputs, packed, out of TMEM
      uint32_t pk[O_COLS / 2];
#pragma unroll
      for (int c = 0; c < O_COLS; c += 32) {
        uint32_t o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
        if (T > 0) {
          tmem_ld_32x32b_x32(t_o + c, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f);
          pk[(c + k) / 2] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
      if (T > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[q]);
      }
      // to memory, 64 bytes of each row at a time: lane l then has bytes 16 (l % 4) of rows 8 k + l / 4
      uint8_t* box = stage_out + (warp - 4) * (32 * C::OUT_PITCH);
      __nv_bfloat16* dst[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = quad * 32 + 8 * k + (lane >> 2), rt = r / args.group;
        const int to = wk.tok0 + q * args.tok_per_tile + rt;
        dst[k] = nullptr;
        if (ok && rt < args.tok_per_tile && to < args.q_len)
          dst[k] = args.out + wk.b * args.out_batch + to * args.out_row +
                   (static_cast<int64_t>(wk.kvh) * args.group + (r - rt * args.group)) * args.out_head + (lane & 3) * 8;
      }
#pragma unroll
      for (int c = 0; c < O_COLS; c += 32) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(box + lane * C::OUT_PITCH + 16 * k) =
              make_uint4(pk[c / 2 + 4 * k], pk[c / 2 + 4 * k + 1], pk[c / 2 + 4 * k + 2], pk[c / 2 + 4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(box + (8 * k + (lane >> 2)) * C::OUT_PITCH + 16 * (lane & 3));
          if (dst[k] != nullptr) *reinterpret_cast<uint4*>(dst[k] + c) = v;
        }
        __syncwarp();
      }
    }
    if (q == 0) named_barrier_sync(1, 256);  // the last turn that was passed on
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// head_dim 256 on CTA pairs (tcgen05 cta_group::2): 256 rows, 128 per CTA.  One CTA per 128 rows would read 128 KB of K and
// V per 128 keys for 2048 cycles of tensor work, more than L2 and shared memory deliver beside the MMAs' own reads: its
// key tile took 3030 cycles (16384 x 1941 x 18 heads: 507 us).  In a pair each CTA loads half: 64 of a tile's 128 keys
// (S, K-major, is split by its columns), and 128 of V's 256 columns (O is split by its columns in the same way).
// Roles and barriers as above with these differences: the leader's MMA warp issues for both CTAs; the loads' bytes of
// both are counted by the leader's `full` and `q_full`; commits arrive in both CTAs; the softmax warps of both
// arrive on the leader's `p_ready` and `o_free`.  16384 x 1941 x 18 heads: 441 us, 1330 TFLOP/s (83% of the measured burst rate);
// 4096 x 512: 45.5 us, where a piece of work has four key tiles and its last products, output and first softmax are in turn.  Where rank 1 has V rows to clear behind a sample's last key, it
// has to see them land, so those loads are counted by a barrier of its own (the leader's MMA then waits for them
// through `p_ready`).
struct AttnPairCfg {
  static constexpr int D = 256;
  static constexpr int BM = 128, BN = 128;                // rows per CTA, keys per tile
  static constexpr int THREADS = 384;
  static constexpr int CHUNK_BYTES = 16384;               // K: 64 keys x 128 elements, V: 64 keys x 128 elements
  static constexpr int CHUNKS = 2;                        // per CTA and key tile, of K and of V
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int AUX_BYTES = 5120;
  static constexpr int OUT_PITCH = 80;
  static constexpr int OUT_BYTES = 8 * 32 * OUT_PITCH;
  static constexpr int STAGES = 8;
  static constexpr int SMEM_BYTES = AUX_BYTES + 1023 + Q_BYTES + STAGES * CHUNK_BYTES + OUT_BYTES;
  static constexpr int S_COL = 256;
  static constexpr uint32_t IDESC_S = idesc_bf16(2 * BM, BN, false);
  static constexpr uint32_t IDESC_O = idesc_bf16(2 * BM, D, true);
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// Whether V rows of key tile t have to be cleared: it holds keys behind the sample's last one that are in memory.
__device__ __forceinline__ bool attn_clears(const AttnArgs& a, const AttnWork& w, int t) {
  return w.len - t * 128 < 128 && w.len < a.kv_len;
}

__global__ void __launch_bounds__(384, 1) __cluster_dims__(2, 1, 1)
    attention_pair_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs args) {
  using C = AttnPairCfg;
  constexpr int D = C::D;
  extern __shared__ uint8_t smem_raw[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw);
  uint64_t* empty = full + C::STAGES;
  uint64_t* q_full = empty + C::STAGES;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;   // [2]
  uint64_t* p_ready = s_full + 2;   // [2]
  uint64_t* o_done = p_ready + 2;
  uint64_t* o_free = o_done + 1;
  uint64_t* v_own = o_free + 1;     // [2]: rank 1: V of a last tile whose rows it clears, in turn
  uint64_t* drain = v_own + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_abort = abort_flag + 1;
  float* row_max = reinterpret_cast<float*>(smem_raw + 512);  // [2 tiles][2 halves][128], then the sums alike
  uint8_t* qs = smem_raw + C::AUX_BYTES;
  qs += (1024u - (smem_u32(qs) & 1023u)) & 1023u;
  uint8_t* ring = qs + C::Q_BYTES;
  uint8_t* stage_out = ring + C::STAGES * C::CHUNK_BYTES;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster = blockIdx.x >> 1, num_clusters = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 16);  // the leader's: the softmax warps of both CTAs
    }
    mbar_init(o_done, 1);
    mbar_init(o_free, 16);         // the leader's
    mbar_init(&v_own[0], 1);
    mbar_init(&v_own[1], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  bool ok = true;

  if (warp < 4) {
    regs_decrease<56>();
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------------- TMA producer (both CTAs)
        int n = 0, w = 0, z = 0;  // chunks issued, pieces of work with keys, last tiles on v_own
        // a chunk: two boxes of 64 elements x 64 keys.  K: keys 64 rank + .. of the tile, 128 elements; V: 64 keys, this
        // CTA's 128 of the 256 elements.  Both CTAs' bytes are counted by the leader's barrier.
        auto load = [&](const CUtensorMap* map, int x, int y, int row, int b, uint64_t* own) {
          const int st = n % C::STAGES;
          if (!mbar_wait(&empty[st], ((n / C::STAGES) & 1) ^ 1, abort_flag, args.timeout_ns)) return false;
          if (rank == 0) mbar_arrive_expect_tx(&full[st], own != nullptr ? C::CHUNK_BYTES : 2 * C::CHUNK_BYTES);
          uint8_t* dst = ring + st * C::CHUNK_BYTES;
          for (int s = 0; s < 2; ++s) {
            if (own != nullptr && rank == 1)
              tma_load_4d(dst + s * (C::CHUNK_BYTES / 2), map, own, x + s * 64, y, row, b);
            else
              tma_load_4d_pair(dst + s * (C::CHUNK_BYTES / 2), map, cluster_addr(&full[st], 0), x + s * 64, y, row, b);
          }
          ++n;
          return true;
        };
        for (int i = cluster; ok && i < args.works; i += num_clusters) {
          const AttnWork wk = attn_work<2>(args, i);
          if (wk.tiles == 0) continue;
          auto load_k = [&](int t) {
            for (int c = 0; ok && c < C::CHUNKS; ++c)
              ok = load(&maps.k, c * 128, wk.kvh * args.kh_mul, t * C::BN + rank * 64, wk.b * args.kb_mul, nullptr);
          };
          auto load_v = [&](int t) {
            // Two barriers in turn: the ring holds the tiles of two pieces of work, so the bytes of one tile can be in
            // before the warps have looked for those of the one before, but not before they have for the one before that.
            uint64_t* own = attn_clears(args, wk, t) ? &v_own[z & 1] : nullptr;
            if (own != nullptr) {
              if (rank == 1) {
                if (z > 1) ok = mbar_wait(own, ((z >> 1) - 1) & 1, abort_flag, args.timeout_ns);
                if (!ok) return;
                mbar_arrive_expect_tx(own, C::CHUNKS * C::CHUNK_BYTES);
              }
              ++z;
            }
            for (int c = 0; ok && c < C::CHUNKS; ++c)
              ok = load(&maps.v, rank * 128, wk.kvh * args.vh_mul, t * C::BN + c * 64, wk.b * args.vb_mul, own);
          };
          // the first keys do not wait for the queries' buffer
          load_k(0);
          if (ok) ok = mbar_wait(q_empty, (w & 1) ^ 1, abort_flag, args.timeout_ns);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(q_full, 2 * args.tok_per_tile * args.group * D * 2);
          for (int s = 0; s < D / 64; ++s)
            tma_load_4d_pair(qs + s * (C::BM * 128), &maps.q, cluster_addr(q_full, 0), s * 64, wk.kvh * args.group,
                             wk.tok0 + rank * args.tok_per_tile, wk.b * args.qb_mul);
          ++w;
          for (int t = 0; ok && t < wk.tiles; ++t) {
            if (t + 1 < wk.tiles) load_k(t + 1);
            load_v(t);
          }
        }
        if (!ok) raise_device_error(args.error_word, kErrTimeout, abort_flag);
        // The copies in flight, as above.  Rank 1's are counted by the leader, which waits here for both CTAs' before the
        // cluster's last barrier; where it gave up before rank 1 did, those of rank 1 that it never armed a barrier
        // for have a whole time limit to land.
        if (rank == 0) {
          bool landed = w == 0 || mbar_wait(q_full, (w - 1) & 1, never_abort, args.timeout_ns);
          for (int i = max(0, n - C::STAGES); landed && i < n; ++i)
            landed = mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, never_abort, args.timeout_ns);
          if (!ok && landed) mbar_wait(&full[n % C::STAGES], (n / C::STAGES) & 1, never_abort, args.timeout_ns);
        } else {
          for (int i = max(0, z - 2); i < z; ++i) mbar_wait(&v_own[i & 1], (i >> 1) & 1, never_abort, args.timeout_ns);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0) {
        // ---------------------------------------------------------------- MMA issuer (leader)
        const uint32_t t_base = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
        const uint64_t q_desc = desc_kmajor_swizzled<128>(smem_u32(qs));
        const uint64_t k_desc = desc_kmajor_swizzled<128>(smem_u32(ring));
        const uint64_t v_desc = desc_mnmajor_sw128(smem_u32(ring), C::CHUNK_BYTES / 2);
        int st = 0, n = 0, w = 0;  // ring position; key tiles and pieces of work done
        uint32_t phase = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, args.timeout_ns));
          tc_fence_after();
          return got;
        };
        auto wait_cluster = [&](uint64_t* bar, uint32_t parity) {
          const bool got = __all_sync(0xFFFFFFFFu, mbar_wait<true>(bar, parity, abort_flag, args.timeout_ns));
          tc_fence_after();
          return got;
        };
        auto advance = [&] {
          tc_commit_pair_warp(&empty[st], 0x3);
          if (++st == C::STAGES) {
            st = 0;
            phase ^= 1u;
          }
        };
        auto issue_s = [&](int buf) {
#pragma unroll
          for (int c = 0; c < C::CHUNKS; ++c) {
            if (!wait(&full[st], phase)) return false;
            const uint64_t kd = k_desc + st * (C::CHUNK_BYTES >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)  // 128 elements: two slices of 64
              tc_mma_bf16_ss_pair_warp(t_base + C::S_COL + buf * C::BN,
                                       q_desc + ((2 * c + k / 4) * (C::BM * 128) >> 4) + 2 * (k % 4),
                                       kd + (k / 4) * (C::CHUNK_BYTES / 2 >> 4) + 2 * (k % 4), C::IDESC_S, c | k);
            advance();
          }
          tc_commit_pair_warp(&s_full[buf], 0x3);
          return true;
        };
        auto issue_o = [&](int buf, int accumulate) {
#pragma unroll
          for (int c = 0; c < C::CHUNKS; ++c) {
            if (!wait(&full[st], phase)) return false;
            const uint64_t vd = v_desc + st * (C::CHUNK_BYTES >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 64 keys
              tc_mma_bf16_ts_pair_warp(t_base, t_base + C::S_COL + buf * C::BN + c * 32 + k * 8, vd + k * (16 * 128 >> 4),
                                       C::IDESC_O, accumulate | c | k);
            advance();
          }
          tc_commit_pair_warp(o_done, 0x3);
          return true;
        };
        for (int i = cluster; ok && i < args.works; i += num_clusters) {
          const AttnWork wk = attn_work<2>(args, i);
          if (wk.tiles == 0) continue;
          ok = wait(q_full, w & 1) && issue_s(n & 1);
          if (wk.tiles == 1) tc_commit_pair_warp(q_empty, 0x3);
          for (int j = 0; ok && j < wk.tiles; ++j, ++n) {
            if (j + 1 < wk.tiles) {
              ok = issue_s((n + 1) & 1);
              if (j + 2 == wk.tiles) tc_commit_pair_warp(q_empty, 0x3);
            }
            if (ok && j == 0) ok = wait(o_free, (w & 1) ^ 1);
            // rank 1's arrivals for a tile whose V rows it cleared publish those zeros, which these MMAs read
            ok = ok && (attn_clears(args, wk, j) ? wait_cluster(&p_ready[n & 1], (n >> 1) & 1) : wait(&p_ready[n & 1], (n >> 1) & 1)) &&
                 issue_o(n & 1, j);
          }
          ++w;
        }
        if (!ok && lane == 0) raise_device_error(args.error_word, kErrTimeout, abort_flag);
        tc_commit_pair_warp(drain, 0x1);
        mbar_wait(drain, 0, never_abort, args.timeout_ns);
      }
      __syncwarp();
    }
  } else {
    regs_increase<224>();
    // -------------------------------------------------------------------- softmax and output
    constexpr int COLS = 64;         // of a key tile, per thread
    constexpr int O_COLS = D / 2;
    const int half = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t t_o = t_lane + half * O_COLS;
    const uint32_t leader_p[2] = {cluster_addr(&p_ready[0], 0), cluster_addr(&p_ready[1], 0)};
    const uint32_t leader_o_free = cluster_addr(o_free, 0);
    const int tok_in = row / args.group, g = row % args.group;
    int n = 0, chunk0 = 0, z = 0;  // key tiles done; ring chunks of the work before; last tiles on v_own
    for (int i = cluster; i < args.works; i += num_clusters) {
      const AttnWork wk = attn_work<2>(args, i);
      const int T = wk.tiles;
      float m = -INFINITY, sum = 0.0f;
      AttnExponent x{};
      for (int j = 0; j < T; ++j, ++n) {
        const int buf = n & 1;
        const uint32_t parity = (n >> 1) & 1;
        const uint32_t t_s = t_lane + C::S_COL + buf * C::BN;
        // a warp whose wait ran out goes on through the barriers of its pair, so that none waits there for good
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[buf], parity, abort_flag, args.timeout_ns));
        tc_fence_after();
        uint32_t raw[COLS];
#pragma unroll
        for (int c = 0; c < COLS; c += 32)
          tmem_ld_32x32b_x32(t_s + half * COLS + c, *reinterpret_cast<uint32_t(*)[32]>(raw + c));
        tmem_ld_wait();
        const int left = wk.len - j * C::BN - half * COLS;  // keys among this thread's columns
        if (left < COLS) {
#pragma unroll
          for (int k = 0; k < COLS; ++k)
            if (k >= left) raw[k] = 0xFF800000u;  // -infinity
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < COLS; k += 2)
          mx4[(k >> 1) & 3] = fmaxf(fmaxf(mx4[(k >> 1) & 3], __uint_as_float(raw[k])), __uint_as_float(raw[k + 1]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        float* mine = row_max + buf * 256;
        mine[half * 128 + row] = mx;
        named_barrier_sync(1 + quad, 64);  // the two warps of these 32 rows; also: both have read their half of S
        mx = fmaxf(mx, mine[(half ^ 1) * 128 + row]);
        if (!ok) continue;
        if (j == 0) {
          m = mx;
          x = attn_exponent(m, args.scale_log2);
        } else {
          const bool grow = (mx - m) * args.scale_log2 > 8.0f;
          if (__any_sync(0xFFFFFFFFu, grow)) {
            // the rows that need it; a neighbour's bits do not depend on them
            const float f = grow ? ex2((m - mx) * args.scale_log2) : 1.0f;
            if (grow) {
              m = mx;
              x = attn_exponent(m, args.scale_log2);
            }
            sum *= f;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_done, (n - 1) & 1, abort_flag, args.timeout_ns));
            if (!ok) continue;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < O_COLS; c += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(t_o + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st_32x32b_x32(t_o + c, o);
            }
            tmem_st_wait();
          }
        }
        const float2 scale2 = make_float2(x.s, x.s), ref2 = make_float2(-x.ref, -x.ref);
        float2 s2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float2 e = fma2(make_float2(__uint_as_float(raw[c + k]), __uint_as_float(raw[c + k + 1])), scale2, ref2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            s2[(k >> 1) & 1] = add2(s2[(k >> 1) & 1], e);
            const __nv_bfloat162 v = __floats2bfloat162_rn(e.x, e.y);
            p[k >> 1] = *reinterpret_cast<const uint32_t*>(&v);
          }
          tmem_st_32x32b_x16(t_s + (half * COLS + c) / 2, p);
        }
        sum += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
        // the last tile's V rows behind the sample's last key
        const bool clears = attn_clears(args, wk, j);
        if (clears) {
          const int keys = wk.len - j * C::BN;
          if (rank == 1)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&v_own[z & 1], (z >> 1) & 1, abort_flag, args.timeout_ns));
          ++z;
          // chunks of this work before V of tile j (its last)
          for (int c = 0; ok && c < C::CHUNKS; ++c) {
            const int at = chunk0 + (2 * j + 1) * C::CHUNKS + c;
            if (rank == 0)
              ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[at % C::STAGES], (at / C::STAGES) & 1, abort_flag, args.timeout_ns));
            if (!ok) break;
            uint8_t* chunk = ring + (at % C::STAGES) * C::CHUNK_BYTES;
            const int from = max(0, keys - c * 64) * 128;  // whole rows: the swizzle stays within a row
            for (int s = 0; s < 2; ++s)
              for (int b = from + (threadIdx.x - 128) * 16; b < C::CHUNK_BYTES / 2; b += 256 * 16)
                *reinterpret_cast<uint4*>(chunk + s * (C::CHUNK_BYTES / 2) + b) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          if (!ok) continue;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
#ifdef NVFP4_TEST_HOOKS
        if (args.test_withhold) continue;
#endif
        if (lane == 0) {
          if (clears) mbar_arrive_release_cluster(leader_p[buf]);
          else mbar_arrive_cluster(leader_p[buf]);
        }
      }
      chunk0 += 2 * T * C::CHUNKS;
      // the phase before the last first, as above
      if (ok && T > 1) ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_done, n & 1, abort_flag, args.timeout_ns));
      if (ok && T > 0) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(o_done, (n - 1) & 1, abort_flag, args.timeout_ns));
        tc_fence_after();
      }
      if (!ok && lane == 0) raise_device_error(args.error_word, kErrTimeout, abort_flag);
      // the row's sum is that of its two halves; two buffers, as a warp may be one piece of work ahead of its partner
      float* mine = row_max + 512 + (i / num_clusters & 1) * 256;
      mine[half * 128 + row] = sum;
      named_barrier_sync(1 + quad, 64);
      sum += mine[(half ^ 1) * 128 + row];
      const int tok = wk.tok0 + rank * args.tok_per_tile + tok_in;
      const bool live = ok && tok_in < args.tok_per_tile && tok < args.q_len;
      const float f = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
      if (live && args.lse != nullptr && half == 0)
        args.lse[(wk.b * static_cast<int64_t>(args.heads) + wk.kvh * args.group + g) * args.q_len + tok] =
            sum == 0.0f ? -INFINITY : __fmaf_rn(m, args.scale_log2, log2f(sum)) * 0.6931471805599453f;
      // the row's outputs, packed, out of TMEM
      uint32_t pk[O_COLS / 2];
#pragma unroll
      for (int c = 0; c < O_COLS; c += 32) {
        uint32_t o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
        if (T > 0) {
          tmem_ld_32x32b_x32(t_o + c, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f);
          pk[(c + k) / 2] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
      if (T > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(leader_o_free);
      }
      // to memory, 64 bytes of each row at a time: lane l then has bytes 16 (l % 4) of rows 8 k + l / 4
      uint8_t* box = stage_out + (warp - 4) * (32 * C::OUT_PITCH);
      __nv_bfloat16* dst[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = quad * 32 + 8 * k + (lane >> 2), rt = r / args.group;
        const int to = wk.tok0 + rank * args.tok_per_tile + rt;
        dst[k] = nullptr;
        if (ok && rt < args.tok_per_tile && to < args.q_len)
          dst[k] = args.out + wk.b * args.out_batch + to * args.out_row +
                   (static_cast<int64_t>(wk.kvh) * args.group + (r - rt * args.group)) * args.out_head + half * O_COLS + (lane & 3) * 8;
      }
#pragma unroll
      for (int c = 0; c < O_COLS; c += 32) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(box + lane * C::OUT_PITCH + 16 * k) =
              make_uint4(pk[c / 2 + 4 * k], pk[c / 2 + 4 * k + 1], pk[c / 2 + 4 * k + 2], pk[c / 2 + 4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(box + (8 * k + (lane >> 2)) * C::OUT_PITCH + 16 * (lane & 3));
          if (dst[k] != nullptr) *reinterpret_cast<uint4*>(dst[k] + c) = v;
        }
        __syncwarp();
      }
    }
  }

  // the leader's MMAs read both CTAs' shared memory and write both TMEMs, and each CTA arrives on the other's barriers
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace nvfp4
