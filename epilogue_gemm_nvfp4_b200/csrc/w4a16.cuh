// The linear of a few rows on NVFP4 weights (W4A16): bf16 activations, in block fixed point, times a stored NVFP4
// weight.  For one to 32 rows the weight's 0.5625 bytes per element are nearly all that moves:
//
//   y[m,n] = g * sum_k x'[m,k] * e2m1(code[n,k]) * e4m3(scale[n, k/16]),   x' = x or silu(x)
//
// Nothing is decoded.  The tensor cores multiply E2M1 by E2M1 with block scales, so x' is written as
// kW4Digits E2M1 tensors, the digits of a fixed-point number of base 8 per 16-element block:
//
//   x'[m,k] = 2^(E_m - 8) * s[m,b] * sum_t 8^-t * d_t[m,k],   d_t in {0, +-0.5, +-1, +-1.5, +-2},  b = k / 16
//
// with s = 2^(e_b - E_m + 8) an E4M3 scale shared by the block's digits, e_b the exponent of the block's largest
// element and E_m that of the row's.  (An integer q = rint(x' 2^16 / 2^e_b), |q| <= 2^17, in digits of -4 .. 4;
// n / 2 has the E2M1 code |n|.)  The weight is the 128-row operand of tcgen05.mma.kind::mxf4nvf4, the digits
// are its columns: digit t of row m is column t * MP + m, and the epilogue adds a row's columns with 8^-t.  Every
// product is exact and summed in fp32.  x' itself is rounded to at most 2^-17 of its block's power of two (2^-34 of the
// row's where a block lies 2^-17 and more below it, the least E4M3 scale): nothing for bf16 elements down to 2^-9 of that
// power, all of an element below 2^-17 of it; silu(x), an fp32 number, is rounded so throughout.  The rounding of
// the bf16 output is 2^-8.
// Measured: one row by [27648 x 4608] 17.1 us (4.2 TB/s of the weight's bytes), 7 rows by the gated [24576 x 4608] 18.5 us,
// 32 rows by [4608 x 53248] 37.1 us (3.8 TB/s), 2 rows by [4608 x 256] 5.3 us.  About 5 us are launches, the first and the last
// kernel.  The stream itself runs at HBM speed up to 16 rows; with 32 the digits (28 KB a chunk beside 36 KB of
// weights) make it one of L2's, at 12 TB/s.
// Decoding the weight for mma.sync instead (E2M1 pair -> f16x2, times the scale) took about 300 instructions per 32 x 128
// weights: 28 us for the one row and 150 us for the 32, bound by instruction issue and the older tensor path.
//
// Kernels, each launched so that it starts while the one before runs, and waits for its end where it needs it:
//   1. the digits (a cluster of CTAs per row), written to the workspace as the shared-memory images of
//      256-element chunks;
//   2. the products, one CTA per SM, which fill their rings with weights before they wait for 1; the sums go to the
//      workspace;
//   3. the outputs: the parts of a sum are added, and the epilogue runs.
// For one or two rows (kFused) every CTA of 2 makes the digits that it needs for itself, in shared memory, and there is no 1.
// (Bringing the weights behind the ring into L2 while the digits are made changed nothing: the stores of the digits, and so the
// end of 1, wait behind that stream.)
// (One cooperative kernel with grid barriers instead of the three: 2 to 3 us more per launch.)
//
// Work of 2.  A unit is 256 weight rows (two MMA row blocks that share the digits' chunk; for the gated SiLU 128
// rows of a and the 128 of b that pair with them), and its chunks of 256 elements; the chunks of all units
// form one line, which is cut into equal ranges, one per CTA: every SM streams the same number of bytes
// whatever N and K are.  The parts of a unit that is cut between CTAs are added in the order of the line.  The cut
// depends on N, K and the number of SMs only, so a row's bits do not depend on the rows that come with it.
//
// Roles in 2: warp 0 producer (TMA and bulk copies into the ring); warp 1 MMA issuer (scales to TMEM by
// tcgen05.cp, which runs in order with the MMAs); warp 2 TMEM; warps 4-11 take the sums out, a warpgroup
// per row block, thread = weight row, with the accumulators double-buffered (up to 16 rows).
#pragma once

#include <cooperative_groups.h>

#include "gemm.cuh"

namespace nvfp4 {

constexpr int kW4MaxRows = 32;
constexpr int kW4Digits = 6;
constexpr int kW4Chunk = 256;     // elements of K per stage
constexpr int kW4MaxCtas = 160;
constexpr int kW4MaxLine = 1 << 30;  // chunks in the line
constexpr int kW4Threads = 384;      // of the product kernel
constexpr int kW4PrepThreads = 512;  // of the digits' kernel
constexpr int kW4FusedRows = 2;
constexpr int kW4FusedChunks = 16;   // rows times chunks of digits that a CTA makes for itself

struct W4Args {
  const __nv_bfloat16* x;
  int64_t ldx;
  int M, N, K, silu;
  const uint8_t* scales;
  int k_atoms;
  const float* g;
  int chunks;             // per unit
  int units;
  int base, rest;         // the line's cut: CTA i has base chunks, the first `rest` CTAs one more
  uint8_t* digits;        // workspace: chunk images
  float* factor;          // [32]: 2^(E_m - 8)
  float* partial;         // [unit + CTA][2][MP][128]
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  int64_t ld_res;
  const float* gate;
  __nv_bfloat16* out;
  int64_t ld_out;
  int kind;
  unsigned int* error_word;
  uint64_t timeout_ns;
#ifdef NVFP4_TEST_HOOKS
  int test_withhold;  // test builds only: accumulators are never given back, so the wait for the next free one runs out
#endif
};

// Columns of the digit operand for MP rows, and the bytes of one chunk image: the columns' codes (128 bytes each, in
// the 128-byte swizzle), then per 64 elements the scale atoms of the columns' 128-row blocks.
__host__ __device__ constexpr int w4_cols(int mp) { return (kW4Digits * mp + 15) / 16 * 16; }
__host__ __device__ constexpr int w4_sf_blocks(int mp) { return (w4_cols(mp) + 127) / 128; }
__host__ __device__ constexpr int w4_image_bytes(int mp) { return w4_cols(mp) * 128 + 4 * w4_sf_blocks(mp) * 512; }

// x * 2^s for any s an exponent difference can give, in two exact steps.
__device__ __forceinline__ float scale_pow2(float x, int s) {
  const int h = s / 2, r = s - h;
  return x * __int_as_float((127 + h) << 23) * __int_as_float((127 + r) << 23);
}

// The exponent of a magnitude given by its fp32 bits; subnormals and zero count as -126, infinities and NaN as 127.
__device__ __forceinline__ int w4_exponent(uint32_t bits) { return min(max(static_cast<int>(bits >> 23), 1), 254) - 127; }

__device__ __forceinline__ void w4_unpack4(const W4Args& a, uint2 w, float (&v)[4]) {
  v[0] = __uint_as_float(w.x << 16);
  v[1] = __uint_as_float(w.x & 0xFFFF0000u);
  v[2] = __uint_as_float(w.y << 16);
  v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  if (a.silu) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = silu(v[i]);
  }
}

// The E2M1 codes of q's digits, digit t (from the top) in nibble t: q = sum_t n_t 8^(5 - t), n_t of -4 .. 4, code |n|
// with the sign in bit 3 (n / 2 in E2M1).
__device__ __forceinline__ uint32_t w4_digits(int q) {
  q += 4 * 4681;  // + 4 in each of the five low digits: they become 0 .. 7, the top one stays -4 .. 4
  const int top = q >> 15;
  // d = n + 4 of the low digits, most significant one in the lowest nibble
  uint32_t d = ((q >> 12) & 7) | ((q >> 5) & 0x70) | ((q << 2) & 0x700) | ((q << 9) & 0x7000) | ((q << 16) & 0x70000);
  const uint32_t neg = (~d >> 2) & 0x11111u;  // n < 0: code 8 | (4 - d); else d - 4
  d = (((d & 0x33333u) ^ (neg * 3u)) + neg) | (neg << 3);
  return (static_cast<uint32_t>(top < 0 ? 8 - top : top) & 15u) | (d << 4);
}

// The largest magnitude of 8 elements of x', as fp32 bits.
__device__ __forceinline__ uint32_t w4_max8(const W4Args& a, uint4 w) {
  if (!a.silu) {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t p = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
    return max(p << 16, p & 0xFFFF0000u);
  }
  float v[4], u[4];
  w4_unpack4(a, make_uint2(w.x, w.y), v);
  w4_unpack4(a, make_uint2(w.z, w.w), u);
  uint32_t b = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    b = max(b, max(__float_as_uint(v[i]) & 0x7FFFFFFFu, __float_as_uint(u[i]) & 0x7FFFFFFFu));
  return b;
}

// The digits of 4 elements of row m, quad j of a chunk, into the chunk's image (a block is four neighbouring lanes of a
// warp, all of which are here).  Rows from M to MP are left as they are: their columns are computed from
// whatever is there and never stored.
template <int MP>
__device__ __forceinline__ void w4_convert4(const W4Args& a, int m, int row_e, uint8_t* image, int j, bool live, uint2 raw) {
  float v[4];
  w4_unpack4(a, raw, v);
  uint32_t bits = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) bits = max(bits, __float_as_uint(v[k]) & 0x7FFFFFFFu);
  bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 1));
  bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 2));
  if (!live) return;
  const int be = max(w4_exponent(bits), row_e - 17);
  const int p = be - row_e + 8;  // 2^p as E4M3: -9 .. 8
  uint32_t sf = p >= -6 ? static_cast<uint32_t>(p + 7) << 3 : 1u << (p + 9);
  if (bits >= 0x7F800000u) sf = 0x7Fu;  // an infinity or NaN: NaN, and so are the row's results
  uint32_t el[4];
  // 2^(16 - be) in two exact factors, as scale_pow2
  const int s1 = (16 - be) / 2, s2 = 16 - be - s1;
  const float f1 = __int_as_float((127 + s1) << 23), f2 = __int_as_float((127 + s2) << 23);
#pragma unroll
  for (int k = 0; k < 4; ++k) el[k] = w4_digits(__float2int_rn(v[k] * f1 * f2));
  // nibble t of the four elements side by side: bytes of digits 0, 2, 4 and 1, 3, 5 of a pair of elements first
  const uint32_t lo[2] = {(el[0] & 0x0F0F0Fu) | ((el[1] & 0x0F0F0Fu) << 4), ((el[0] >> 4) & 0x0F0F0Fu) | (el[1] & 0xF0F0F0u)};
  const uint32_t hi[2] = {(el[2] & 0x0F0F0Fu) | ((el[3] & 0x0F0F0Fu) << 4), ((el[2] >> 4) & 0x0F0F0Fu) | (el[3] & 0xF0F0F0u)};
  // column t * MP + m: its code row, 2 bytes of quad j in the swizzle, and its place in the scale atoms, block j / 4.
  // MP and t are known here, so the columns of a row are constant offsets apart.
  uint8_t* codes = image + m * 128 + (j & 7) * 2;
  uint8_t* scales = image + w4_cols(MP) * 128 + (j >> 4) * w4_sf_blocks(MP) * 512 + m * 16 + ((j >> 2) & 3);
#pragma unroll
  for (int t = 0; t < kW4Digits; ++t) {
    const int c0 = t * MP;  // of row 0; rows stay within a group of 32 columns
    const int sw = MP % 8 == 0 ? m & 7 : (c0 + m) & 7;
    *reinterpret_cast<uint16_t*>(codes + c0 * 128 + (((j >> 3) ^ sw) << 4)) =
        static_cast<uint16_t>(__byte_perm(lo[t & 1], hi[t & 1], (t >> 1) | (4 + (t >> 1)) << 4));
    if ((j & 3) == 0) scales[(c0 >> 7) * 512 + (c0 & 31) * 16 + ((c0 >> 5) & 3) * 4] = static_cast<uint8_t>(sf);
  }
}

// One cluster per row: the row's largest exponent, then its digits, 4 elements per thread and step.
template <int MP>
__global__ void __launch_bounds__(kW4PrepThreads) w4a16_prepare_kernel(const __grid_constant__ W4Args a) {
  namespace cg = cooperative_groups;
  __shared__ uint32_t warp_max[kW4PrepThreads / 32];
  __shared__ uint32_t cta_max;
  const cg::cluster_group cluster = cg::this_cluster();
  const int S = static_cast<int>(cluster.num_blocks());
  const int m = blockIdx.x / S;
  const int first = static_cast<int>(cluster.block_rank()) * kW4PrepThreads + threadIdx.x, step = S * kW4PrepThreads;
  const int quads = a.K / 4;  // a multiple of 16: a block's four lanes are in range together
  const uint2* quad = reinterpret_cast<const uint2*>(a.x + m * a.ldx);
  // The product kernel starts its stream of weights at once, or, where reading the row takes longer than that start, when the
  // row is here: beside that stream a read takes microseconds (16 rows, N = 4608: K = 18432 16.1 us at once and 16.9 us
  // later, K = 53248 35.8 and 33.7 us).
  const bool long_row = quads > 2 * step;
  if (!long_row) asm volatile("griddepcontrol.launch_dependents;");
  // the first steps' elements stay in registers, for the same reason
  constexpr int kKeep = 7;
  uint2 keep[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    keep[k] = make_uint2(0u, 0u);
    if (first + k * step < quads) keep[k] = quad[first + k * step];
  }
  uint32_t e = 0u;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    if (k * step >= quads) break;  // uniform
    e = max(e, w4_max8(a, make_uint4(keep[k].x, keep[k].y, 0u, 0u)));
  }
  for (int i = first + kKeep * step; i < quads; i += step) e = max(e, w4_max8(a, make_uint4(quad[i].x, quad[i].y, 0u, 0u)));
  e = __reduce_max_sync(0xFFFFFFFFu, e);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = e;
  __syncthreads();
  if (long_row) asm volatile("griddepcontrol.launch_dependents;");
  e = __reduce_max_sync(0xFFFFFFFFu, warp_max[threadIdx.x & (kW4PrepThreads / 32 - 1)]);
  if (S > 1) {
    if (threadIdx.x == 0) cta_max = e;
    cluster_sync();
    e = __reduce_max_sync(0xFFFFFFFFu, *cluster.map_shared_rank(&cta_max, (threadIdx.x & 31) % S));
  }
  const int row_e = w4_exponent(e);
  if (first == 0) a.factor[m] = scale_pow2(1.0f, row_e - 8);
  // whole warps go round, so that the shuffles have all lanes
  auto convert = [&](int i, uint2 raw) {
    w4_convert4<MP>(a, m, row_e, a.digits + static_cast<int64_t>(i >> 6) * w4_image_bytes(MP), i & 63, i < quads, raw);
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    if (((first + k * step) & ~31) >= quads) break;
    convert(first + k * step, keep[k]);
  }
  for (int i = first + kKeep * step; (i & ~31) < quads; i += step) convert(i, i < quads ? quad[i] : make_uint2(0u, 0u));
  if (S > 1) {
    __syncwarp();
    cluster_sync();  // no CTA leaves while its maximum is read
  }
}

// kFused: the digits of `count` chunks from chunk c0 (of the unit, in turn) into shared memory, image by image, by the
// threads of one CTA; `weights` starts the ring's first loads, behind this CTA's first reads (in front of them it
// would make each take microseconds).
template <int MP, typename Weights>
__device__ __forceinline__ void w4_prepare_own(const W4Args& a, int c0, int count, uint8_t* images, uint32_t* warp_max,
                                               Weights weights) {
  const int octs = a.K / 8;
  int row_e[kW4FusedRows];
  for (int m = 0; m < a.M; ++m) {
    const uint4* oct = reinterpret_cast<const uint4*>(a.x + m * a.ldx);
    uint32_t e = 0u;
    for (int base = 0; base < octs; base += 4 * kW4Threads) {
      uint4 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = base + k * kW4Threads + threadIdx.x;
        w[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i < octs) w[k] = oct[i];
      }
      if (m == 0 && base == 0) weights();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (base + k * kW4Threads >= octs) break;  // uniform
        e = max(e, w4_max8(a, w[k]));
      }
    }
    e = __reduce_max_sync(0xFFFFFFFFu, e);
    if ((threadIdx.x & 31) == 0) warp_max[m * 16 + (threadIdx.x >> 5)] = e;
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kW4FusedRows; ++m) {
    row_e[m] = w4_exponent(__reduce_max_sync(0xFFFFFFFFu, warp_max[m * 16 + (threadIdx.x & 31) % (kW4Threads / 32)]));
    if (m < a.M && blockIdx.x == 0 && threadIdx.x == 0) a.factor[m] = scale_pow2(1.0f, row_e[m] - 8);
  }
  // a warp's 32 quads are half a chunk
  for (int i = threadIdx.x; i < count * 64 * a.M; i += kW4Threads) {
    const int m = i >= count * 64 ? 1 : 0, k = (i - m * count * 64) >> 6, j = i & 63;
    const int c = c0 + k < a.chunks ? c0 + k : c0 + k - a.chunks;
    const int q = c * 64 + j;
    const uint2* quad = reinterpret_cast<const uint2*>(a.x + m * a.ldx);
    const bool live = q < a.K / 4;
    w4_convert4<MP>(a, m, row_e[m], images + k * w4_image_bytes(MP), j, live, live ? quad[q] : make_uint2(0u, 0u));
  }
}

template <int MP, bool kFused>
struct W4Cfg {
  static constexpr int COLS = w4_cols(MP);
  static constexpr int SFB = w4_sf_blocks(MP);
  static constexpr int W_CODES = 128 * 128, W_SCALES = 2048;  // per row block
  static constexpr int IMAGE = w4_image_bytes(MP);
  // stage: codes of both row blocks, digit codes, scales of both, digit scales
  // (kFused: no digits there, their images stay behind the ring)
  static constexpr int X_OFF = 2 * W_CODES, S_OFF = X_OFF + (kFused ? 0 : COLS * 128), XS_OFF = S_OFF + 2 * W_SCALES;
  static constexpr int STAGE_BYTES = XS_OFF + (kFused ? 0 : 4 * SFB * 512);
  static constexpr int OWN_BYTES = kFused ? kW4FusedChunks * IMAGE : 0;
  static constexpr int AUX_BYTES = 1024;
  static constexpr int FIT = (232448 - AUX_BYTES - 1023 - OWN_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  static constexpr int SMEM_BYTES = AUX_BYTES + 1023 + STAGES * STAGE_BYTES + OWN_BYTES;
  static constexpr int BUFS = MP <= 16 ? 2 : 1;               // accumulators of a unit in TMEM
  static constexpr int SLOT_COLS = 32 + 16 * SFB;             // TMEM scale columns of a stage
  static constexpr int SF_COL = BUFS * 2 * COLS;
  static constexpr uint32_t IDESC = idesc_nvf4(128, COLS);
  static_assert(STAGES >= 3 && COLS % 16 == 0 && COLS <= 256, "stages, MMA columns");
  static_assert(SF_COL + 2 * SLOT_COLS <= 512, "TMEM columns");
  static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms stay 1024-byte aligned");
};

// The line of chunks: CTA i has [cut(i), cut(i + 1)).
__device__ __forceinline__ int w4_cut(const W4Args& a, int i) { return i * a.base + min(i, a.rest); }

// The CTA that has chunk `at`.
__device__ __forceinline__ int w4_owner(const W4Args& a, int at) {
  const int head = a.rest * (a.base + 1);
  return at < head ? at / (a.base + 1) : a.rest + (at - head) / a.base;
}

template <int MP, bool kFused>
__global__ void __launch_bounds__(640, 1)  // 96 registers for its 384 threads: CTAs of the other kernels fit beside it
    w4a16_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ W4Args a) {
  using C = W4Cfg<MP, kFused>;
  extern __shared__ uint8_t w4_smem[];
  asm volatile("griddepcontrol.launch_dependents;");
  uint64_t* full = reinterpret_cast<uint64_t*>(w4_smem);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_abort = abort_flag + 1;
  uint32_t* warp_max = reinterpret_cast<uint32_t*>(w4_smem + 512);  // [2][16]
  uint8_t* ring = w4_smem + C::AUX_BYTES;
  ring += (1024u - (smem_u32(ring) & 1023u)) & 1023u;
  uint8_t* own = ring + C::STAGES * C::STAGE_BYTES;  // kFused: this CTA's images, from its first chunk's

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool gated = a.kind == kEpiGatedSilu;
  const int cta = blockIdx.x;
  const int i0 = w4_cut(a, cta), i1 = w4_cut(a, cta + 1);

  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmap);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  bool ok = true;
  const int last_block = (a.N + 127) / 128 - 1;
  auto load_w = [&](int u, int c, int st) {
    const int rb[2] = {gated ? u : 2 * u, gated ? u + a.N / 256 : 2 * u + 1};
    const uint32_t sf = static_cast<uint32_t>(min(4, a.k_atoms - 4 * c)) * 512u;
    const bool two = rb[1] <= last_block;  // an odd last row block: the other half's codes read as zeros
    uint8_t* dst = ring + st * C::STAGE_BYTES;
    mbar_arrive_expect_tx(&full[st], 2 * C::W_CODES + (kFused ? 0 : C::IMAGE) + (two ? 2 * sf : sf));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tma_load_2d(dst + h * C::W_CODES, &tmap, &full[st], c * (kW4Chunk / 2), rb[h] * 128);
      if (h == 0 || two)
        bulk_load(dst + C::S_OFF + h * C::W_SCALES, a.scales + (static_cast<int64_t>(rb[h]) * a.k_atoms + 4 * c) * 512, sf,
                  &full[st]);
    }
  };
  auto load_x = [&](int c, int st) {
    const uint8_t* image = a.digits + static_cast<int64_t>(c) * C::IMAGE;
    uint8_t* dst = ring + st * C::STAGE_BYTES;
    bulk_load(dst + C::X_OFF, image, C::COLS * 128, &full[st]);
    bulk_load(dst + C::XS_OFF, image + C::COLS * 128, 4 * C::SFB * 512, &full[st]);
  };
  const int u0 = i0 / a.chunks, c0 = i0 - u0 * a.chunks;
  const int ahead = min(C::STAGES, i1 - i0);
  int u = u0, c = c0;
  auto next = [&] {
    if (++c == a.chunks) {
      c = 0;
      ++u;
    }
  };

  // the weights do not depend on the digits
  auto first_weights = [&] {
    if (threadIdx.x == 0) {
      for (int i = 0; i < ahead; ++i, next()) load_w(u, c, i);
      u = u0;
      c = c0;
    }
    __syncwarp();
  };
  if constexpr (kFused) {
    w4_prepare_own<MP>(a, c0, min(a.chunks, i1 - i0), own, warp_max, first_weights);
    fence_proxy_async_smem();  // the MMAs read the images
  } else {
    first_weights();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------------ producer
      if (!kFused) {
        asm volatile("griddepcontrol.wait;\n\tfence.proxy.async;" ::: "memory");
        for (int i = 0; i < ahead; ++i, next()) load_x(c, i);
      } else {
        for (int i = 0; i < ahead; ++i) next();
      }
      int st = ahead == C::STAGES ? 0 : ahead, n = ahead;
      uint32_t phase = 0;
      for (; i0 + n < i1; ++n, next()) {
        if (!mbar_wait(&empty[st], phase, abort_flag, a.timeout_ns)) {
          ok = false;
          break;
        }
        load_w(u, c, st);
        if (!kFused) load_x(c, st);
        if (++st == C::STAGES) {
          st = 0;
          phase ^= 1u;
        }
      }
      if (!ok) raise_device_error(a.error_word, kErrTimeout, abort_flag);
      // The copies in flight write this CTA's shared memory: wait for them before it ends.  Whatever became of the others:
      // the MMA warp, which waits for the same copies, may have given up.
      for (int i = max(0, n - C::STAGES); i < n; ++i)
        if (!mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, never_abort, a.timeout_ns)) break;
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------------- MMA issuer
    const uint32_t t_base = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
    const uint64_t w_desc0 = desc_kmajor_swizzled<128>(smem_u32(ring));
    const uint64_t sf_desc0 = desc_scale_atom(smem_u32(ring + C::S_OFF));
    const uint64_t own_desc = desc_kmajor_swizzled<128>(smem_u32(own));
    const uint64_t own_sf_desc = desc_scale_atom(smem_u32(own + C::COLS * 128));
    int st = 0, buf = 0, slot = 0;
    uint32_t phase = 0, acc_phase = 0;
    for (int i = i0; ok && i < i1;) {
      // the chunks of one unit
      const int end = min(i1, i + a.chunks - c);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_empty[buf], acc_phase ^ 1u, abort_flag, a.timeout_ns));
      tc_fence_after();
      const uint32_t d = t_base + buf * 2 * C::COLS;
      uint32_t accumulate = 0;
      for (; ok && i < end; ++i, ++c) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[st], phase, abort_flag, a.timeout_ns));
        if (!ok) break;
        tc_fence_after();
        const uint64_t w_desc = w_desc0 + st * (C::STAGE_BYTES >> 4);
        const uint64_t sf_desc = sf_desc0 + st * (C::STAGE_BYTES >> 4);
        // the chunk's digits and their scales
        const int k_own = c >= c0 ? c - c0 : c - c0 + a.chunks;
        const uint64_t x_desc = kFused ? own_desc + k_own * (C::IMAGE >> 4) : w_desc + (C::X_OFF >> 4);
        const uint64_t xs_desc = kFused ? own_sf_desc + k_own * (C::IMAGE >> 4) : sf_desc + ((C::XS_OFF - C::S_OFF) >> 4);
        const uint32_t sfa = t_base + C::SF_COL + slot * C::SLOT_COLS, sfb = sfa + 32;
        const int ks = min(4, a.k_atoms - 4 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= ks) break;  // uniform
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tc_cp_32x128b_warpx4_warp(sfa + 16 * h + 4 * k, sf_desc + ((h * C::W_SCALES + k * 512) >> 4));
#pragma unroll
          for (int j = 0; j < C::SFB; ++j)
            tc_cp_32x128b_warpx4_warp(sfb + 4 * (k * C::SFB + j),
                                      xs_desc + ((k * C::SFB + j) * 512 >> 4));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k >= ks) break;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tc_mma_nvf4_warp(d + h * C::COLS, w_desc + h * (C::W_CODES >> 4) + 2 * k, x_desc + 2 * k, C::IDESC,
                             accumulate | k, sfa + 16 * h + 4 * k, sfb + 4 * k * C::SFB);
        }
        accumulate = 1;
        tc_commit_warp(&empty[st]);
        slot ^= 1;
        if (++st == C::STAGES) {
          st = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (c == a.chunks) c = 0;
      tc_commit_warp(&acc_full[buf]);
      if (++buf == C::BUFS) {
        buf = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok && lane == 0) raise_device_error(a.error_word, kErrTimeout, abort_flag);
    tc_commit_warp(drain);
    mbar_wait(drain, 0, never_abort, a.timeout_ns);
  } else if (warp >= 4) {
    // -------------------------------------------------------------------- sums to the workspace
    const int h = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(row & 96) << 16) + h * C::COLS;
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int i = i0; i < i1; ++u) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[buf], acc_phase, abort_flag, a.timeout_ns));
      if (!ok) {
        if (lane == 0) raise_device_error(a.error_word, kErrTimeout, abort_flag);
        break;
      }
      tc_fence_after();
      float* part = a.partial + (static_cast<int64_t>(u + cta) * 2 + h) * (MP * 128) + row;
      const uint32_t t_acc = t_lane + buf * 2 * C::COLS;
      constexpr int R = MP < 8 ? MP : 8;  // rows at a time
#pragma unroll
      for (int m0 = 0; m0 < MP; m0 += R) {
        if (m0 >= a.M) break;
        float y[R] = {};
        if constexpr (MP < 8) {
          uint32_t d[16];
          tmem_ld_32x32b_x8(t_acc, d);
          tmem_ld_32x32b_x8(t_acc + 8, d + 8);
          tmem_ld_wait();
#pragma unroll
          for (int t = kW4Digits - 1; t >= 0; --t)
#pragma unroll
            for (int m = 0; m < R; ++m) y[m] = __fmaf_rn(y[m], 0.125f, __uint_as_float(d[t * MP + m]));
        } else {
#pragma unroll
          for (int t = kW4Digits - 1; t >= 0; --t) {
            uint32_t d[8];
            tmem_ld_32x32b_x8(t_acc + t * MP + m0, d);
            tmem_ld_wait();
#pragma unroll
            for (int m = 0; m < R; ++m) y[m] = __fmaf_rn(y[m], 0.125f, __uint_as_float(d[m]));
          }
        }
#pragma unroll
        for (int m = 0; m < R; ++m)
          if (m0 + m < a.M) __stcg(part + (m0 + m) * 128, y[m]);
      }
      tc_fence_before();
      __syncwarp();
#ifdef NVFP4_TEST_HOOKS
      if (lane == 0 && !a.test_withhold) mbar_arrive(&acc_empty[buf]);
#else
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
#endif
      if (++buf == C::BUFS) {
        buf = 0;
        acc_phase ^= 1u;
      }
      i = min(i1, (u + 1) * a.chunks);
    }
  }
  __syncwarp();

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Add the parts of every unit in the order of the line and run the epilogue: a warp has 128 columns of a row.
template <int MP>
__global__ void __launch_bounds__(128) w4a16_finish_kernel(const __grid_constant__ W4Args a) {
  const bool gated = a.kind == kEpiGatedSilu;
  const int lane = threadIdx.x & 31;
  const int halves = gated ? 1 : 2, n_out = gated ? a.N / 2 : a.N;
  const float g = *a.g;
  const bool vec = (a.ld_out & 3) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0 && (n_out & 3) == 0;
  const int task = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (task < a.units * halves * a.M) {
    const int m = task / (a.units * halves), uh = task - m * (a.units * halves);
    const int ou = gated ? uh : uh >> 1, h = gated ? 0 : uh & 1;
    const int n0 = uh * 128 + lane * 4;
    const int first = w4_owner(a, ou * a.chunks), last = w4_owner(a, (ou + 1) * a.chunks - 1);
    const float* p = a.partial + ((static_cast<int64_t>(ou + first) * 2 + h) * MP + m) * 128 + lane * 4;
    float y[4] = {}, y2[4] = {}, b1[4] = {}, b2[4] = {}, res[4] = {}, gate[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = n0 + k;
      if (n >= n_out) break;
      if (a.bias) b1[k] = __bfloat162float(a.bias[n]);
      if (a.bias && gated) b2[k] = __bfloat162float(a.bias[n + n_out]);
      if (a.kind == kEpiResidGate) {
        gate[k] = a.gate[n];
        res[k] = __bfloat162float(a.residual[m * a.ld_res + n]);
      }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what follows is the product kernel's
    const float f = __ldcg(a.factor + m);
    // parts at a time, all loads of which are on their way together
    constexpr int kParts = 6;
    for (int k = first; k <= last; k += kParts, p += kParts * 2 * MP * 128) {
      float4 v[kParts], w[kParts];
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        if (k + i <= last) v[i] = __ldcg(reinterpret_cast<const float4*>(p + i * 2 * MP * 128));
        if (gated && k + i <= last) w[i] = __ldcg(reinterpret_cast<const float4*>(p + (i * 2 + 1) * MP * 128));
      }
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        if (k + i > last) break;
        y[0] += v[i].x, y[1] += v[i].y, y[2] += v[i].z, y[3] += v[i].w;
        if (gated) y2[0] += w[i].x, y2[1] += w[i].y, y2[2] += w[i].z, y2[3] += w[i].w;
      }
    }
    __nv_bfloat16 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v = __fadd_rn(__fmul_rn(__fmul_rn(y[k], g), f), b1[k]);
      if (gated) v = silu(v) * __fadd_rn(__fmul_rn(__fmul_rn(y2[k], g), f), b2[k]);
      else if (a.kind == kEpiResidGate) v = __fmaf_rn(gate[k], v, res[k]);
      o[k] = __float2bfloat16_rn(v);
    }
    __nv_bfloat16* out = a.out + m * a.ld_out + n0;
    if (vec && n0 < n_out) {
      const __nv_bfloat162 lo(o[0], o[1]), hi(o[2], o[3]);
      *reinterpret_cast<uint2*>(out) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (n0 + k < n_out) out[k] = o[k];
    }
  }
}

}  // namespace nvfp4
