// Entry point of the attention to an encoder's states.  Included at the end of nvfp4_api.cu, whose helpers
// (argument checks, per-device state, tensor-map encoder) it uses.
#pragma once

#include "attention.cuh"

namespace {

// 4-D TMA map of a [batch, rows, heads, D] bf16 tensor with any strides: dimensions D, heads, rows, batch, box
// of 64 elements (the 128-byte swizzle) x box_heads x box_rows.  A dimension of stride 0 is mapped with
// extent 1 (the kernel then stays at its coordinate 0).
nvfp4_status make_attn_map(CUtensorMap* map, const void* p, int D, int64_t heads, int64_t rows, int64_t batch,
                           const int64_t* stride, int box_heads, int box_rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return NVFP4_ERR_CUDA;
  const int64_t n[3] = {heads, rows, batch}, s[3] = {stride[2], stride[1], stride[0]};
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D)};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) {
    const bool one = n[i] == 1 || s[i] == 0;
    dims[i + 1] = one ? 1 : static_cast<cuuint64_t>(n[i]);
    strides[i] = static_cast<cuuint64_t>(one ? D : s[i]) * 2;
  }
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}

// Strides of one [batch, rows, heads, D] operand: {batch, row, head}; those of extents of 1 are not read.
nvfp4_status check_attn_strides(const int64_t* s, int64_t batch, int64_t rows, int64_t heads, int D, bool may_broadcast,
                                bool batch_may_broadcast) {
  const int64_t n[3] = {batch, rows, heads};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (s[i] == 0 && ((i == 0 && batch_may_broadcast) || (i == 2 && may_broadcast))) continue;
    if (s[i] < D || s[i] >= (int64_t(1) << 39)) return NVFP4_ERR_INVALID_ARG;  // a byte stride is below 2^40
    if (s[i] % 8) return NVFP4_ERR_MISALIGNED;
  }
  return NVFP4_OK;
}

// The clusters of each size that can be resident at once, of the few-rows kernel (a GPC's SMs left over by clusters of s
// stay idle: 36 clusters of 4 do not fit the 148 SMs in one round).
template <int D>
nvfp4_status attn_resident(DeviceState* st, const int** resident) {
  using C = AttnCfg<D>;
  std::lock_guard<std::mutex> lock(g_mutex);
  int* n = st->attn_clusters[D / 128];
  *resident = n;
  if (n[1] != 0) return NVFP4_OK;
  if (cudaFuncSetAttribute(attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  for (int s = 2; s <= kAttnMaxSplit; ++s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(s * (st->sm_count / s)));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(s);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n[s], attention_kernel<D>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_CUDA;
    }
  }
  n[1] = st->sm_count;
  return NVFP4_OK;
}

// CTAs per cluster that share the key tiles of one query tile: the fewest with which a CTA's share is least, of those
// whose clusters are all resident at once.
int attn_split(const int* resident, int64_t ctas, int64_t kv_len) {
  const int64_t tiles = (kv_len + 127) / 128;
  int best = 1;
  for (int s = 2; s <= kAttnMaxSplit; ++s)
    if (ctas <= resident[s] && (tiles + s - 1) / s < (tiles + best - 1) / best) best = s;
  return best;
}

template <int D>
nvfp4_status launch_attention(const AttnMaps& maps, const AttnArgs& a, dim3 grid, int split, cudaStream_t s) {
  using C = AttnCfg<D>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attention_kernel<D>, maps, a) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_CUDA;
  }
  return launch_status();
}

template <int D>
nvfp4_status launch_attention_rows(DeviceState* st, const AttnMaps& maps, const AttnArgs& a, cudaStream_t s) {
  using C = AttnRowsCfg<D>;
  auto kernel = attention_rows_kernel<D>;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    bool& attr = st->smem_attr_set_attn_rows[D / 128];
    if (!attr) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
        return NVFP4_ERR_CUDA;
      attr = true;
    }
  }
  const int grid = a.works < st->sm_count ? a.works : st->sm_count;
  kernel<<<grid, C::THREADS, C::SMEM_BYTES, s>>>(maps, a);
  return launch_status();
}

// CTA pairs that can be resident at once: the persistent grid must not exceed one wave.
nvfp4_status attn_pairs(DeviceState* st, int* pairs) {
  using C = AttnPairCfg;
  std::lock_guard<std::mutex> lock(g_mutex);
  int& cached = st->attn_pair_clusters;
  if (cached == 0) {
    if (cudaFuncSetAttribute(attention_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
      return NVFP4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (st->sm_count / 2));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, attention_pair_kernel, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return NVFP4_ERR_CUDA;
    }
    cached = n;
  }
  *pairs = cached;
  return NVFP4_OK;
}

nvfp4_status launch_attention_pair(const AttnMaps& maps, const AttnArgs& a, int pairs, cudaStream_t s) {
  using C = AttnPairCfg;
  attention_pair_kernel<<<2 * (a.works < pairs ? a.works : pairs), C::THREADS, C::SMEM_BYTES, s>>>(maps, a);
  return launch_status();
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_cross_attention(const nvfp4_attention_desc* d, nvfp4_stream_t stream) {
  if (!d || d->batch < 0 || d->q_len < 0 || d->kv_len < 0 || d->heads < 1 || d->kv_heads < 1) return NVFP4_ERR_INVALID_ARG;
  if (!(d->scale > 0.0f && d->scale <= 1.0e38f)) return NVFP4_ERR_INVALID_ARG;
  const int D = d->head_dim;
  if ((D != 64 && D != 128 && D != 256) || d->heads % d->kv_heads || d->heads / d->kv_heads > 128 ||
      d->kv_heads > 65535 || d->batch > 65535 || d->q_len > (int64_t(1) << 30) || d->kv_len > (int64_t(1) << 30))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (d->batch == 0 || d->q_len == 0) return NVFP4_OK;
  const int64_t qs[3] = {d->q_batch_stride, d->q_row_stride, d->q_head_stride};
  const int64_t ks[3] = {d->k_batch_stride, d->k_row_stride, d->k_head_stride};
  const int64_t vs[3] = {d->v_batch_stride, d->v_row_stride, d->v_head_stride};
  const int64_t os[3] = {d->out_batch_stride, d->out_row_stride, d->out_head_stride};
  if (!d->q || !d->out || (d->kv_len > 0 && (!d->k || !d->v))) return NVFP4_ERR_INVALID_ARG;
  if (nvfp4_status e = check_attn_strides(qs, d->batch, d->q_len, d->heads, D, false, true)) return e;
  if (nvfp4_status e = check_attn_strides(os, d->batch, d->q_len, d->heads, D, false, false)) return e;
  if (d->kv_len > 0) {
    if (nvfp4_status e = check_attn_strides(ks, d->batch, d->kv_len, d->kv_heads, D, true, true)) return e;
    if (nvfp4_status e = check_attn_strides(vs, d->batch, d->kv_len, d->kv_heads, D, true, true)) return e;
  }
  if (!aligned16(d->q) || !aligned16(d->out) || !aligned16(d->k) || !aligned16(d->v) ||
      (d->kv_lens && !aligned4(d->kv_lens)) || (d->lse && !aligned4(d->lse)))
    return NVFP4_ERR_MISALIGNED;
  DeviceState* st;
  if (nvfp4_status e = device_state(&st)) return e;
  AttnArgs a{};
  a.q_len = static_cast<int>(d->q_len);
  a.kv_len = static_cast<int>(d->kv_len);
  a.group = d->heads / d->kv_heads;
  a.tok_per_tile = 128 / a.group;
  a.qb_mul = qs[0] != 0 || d->batch == 1;
  a.kb_mul = ks[0] != 0;
  a.kh_mul = ks[2] != 0;
  a.vb_mul = vs[0] != 0;
  a.vh_mul = vs[2] != 0;
  a.kv_lens = d->kv_lens;
  a.scale_log2 = d->scale * 1.4426950408889634f;
  a.out = static_cast<__nv_bfloat16*>(d->out);
  a.out_batch = os[0];
  a.out_row = os[1];
  a.out_head = os[2];
  a.lse = d->lse;
  a.heads = d->heads;
  a.error_word = st->error_word;
  a.timeout_ns = wait_timeout_ns();
#ifdef NVFP4_TEST_HOOKS
  a.test_withhold = g_test_withhold_arrivals.load();
#endif
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Tiles of 128 rows, one per CTA with the keys split over clusters while there is room; or the persistent kernels' pieces
  // of two tiles.  The latter need less time for two tiles than the former for two in turn, but more than for one:
  // a piece takes 1.1 to 1.5 times as long as a tile on its CTA (head_dim 128: 64 keys 10.7 and 9.5 us, 512 keys 16.4 and 12.9,
  // 1941 keys 40.7 and 26.9), and on a CTA pair (head_dim 256) 0.9 to 1 times (64 keys 12.9 and 13.2, 1941 keys 33.4 and 38.1).
  // So the rounds of both are compared.  Pieces and tiles, inputs larger than L2 in all:
  //   18 heads of 128: 1280 rows (1 round of pieces, 2 of tiles) 128 keys 10.5 and 15.8 us, 1941 keys 40.8 and 49.7;
  //     3 samples of 600 (2, 2) 15.8 and 16.6, 76 and 50; 2560 (2, 3) 16.4 and 23.3, 77 and 74; 4096 (2, 4) 16.6 and 30.6, 77 and 99;
  //   24 heads of 64: 1280 (1, 2) 128 keys 8.5 and 12.5, 1941 keys 31.8 and 45.0; 3 x 600 (2, 3) 12.1 and 17.9, 58 and 66;
  //     4096 (3, 6) 15.8 and 32.5, 85 and 129;
  //   18 heads of 256, rounds of pairs: 1280 (2, 2) 128 keys 18.4 and 21.7, 1941 keys 57.8 and 70.9; 3 x 600 (3, 2) 23.0 and
  //     23.3, 84 and 73.6; 4096 (4, 4) 30.3 and 43.0, 118 and 143.
  const int64_t rows_per_work = 2 * static_cast<int64_t>(a.tok_per_tile);
  const int64_t q_works = (d->q_len + rows_per_work - 1) / rows_per_work, works = q_works * d->kv_heads * d->batch;
  if (works > (int64_t(1) << 30)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t q_tiles = (d->q_len + a.tok_per_tile - 1) / a.tok_per_tile, tiles = q_tiles * d->kv_heads * d->batch;
  const int* resident = nullptr;
  int pairs = 0;
  if (nvfp4_status e = D == 256 ? attn_resident<256>(st, &resident)
                       : D == 128 ? attn_resident<128>(st, &resident) : attn_resident<64>(st, &resident))
    return e;
  if (D == 256)
    if (nvfp4_status e = attn_pairs(st, &pairs)) return e;
  const int split = attn_split(resident, tiles, d->kv_len);
  const int64_t tile_rounds = (tiles + st->sm_count - 1) / st->sm_count;
  const bool many = split > 1 || tiles == works ? false
                    : D == 256 ? (works + pairs - 1) / pairs <= tile_rounds
                               : 3 * ((works + st->sm_count - 1) / st->sm_count) <= 2 * tile_rounds;
  // keys per box of K and of V: in the pair kernel each CTA has 64 of a tile's keys and of a V chunk's
  const int k_box = many && D == 256 ? 64 : 128, v_box = many && D == 256 ? 64 : 128 / (D / 64);
  AttnMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (nvfp4_status e = make_attn_map(&maps.q, d->q, D, d->heads, d->q_len, d->batch, qs, a.group, a.tok_per_tile))
    return e;
  // no keys: the kernel loads nothing; its maps describe q instead of what is not there
  const bool keys = d->kv_len > 0;
  if (nvfp4_status e = make_attn_map(&maps.k, keys ? d->k : d->q, D, d->kv_heads, keys ? d->kv_len : 1, d->batch,
                                     keys ? ks : qs, 1, k_box))
    return e;
  if (nvfp4_status e = make_attn_map(&maps.v, keys ? d->v : d->q, D, d->kv_heads, keys ? d->kv_len : 1, d->batch,
                                     keys ? vs : qs, 1, v_box))
    return e;
  if (many) {
    a.q_works = static_cast<int>(q_works);
    a.kv_heads = d->kv_heads;
    a.works = static_cast<int>(works);
    if (D == 256) return launch_attention_pair(maps, a, pairs, s);
    if (D == 128) return launch_attention_rows<128>(st, maps, a, s);
    return launch_attention_rows<64>(st, maps, a, s);
  }
  const dim3 grid(static_cast<unsigned>(q_tiles * split), d->kv_heads, static_cast<unsigned>(d->batch));
  if (D == 256) return launch_attention<256>(maps, a, grid, split, s);
  if (D == 128) return launch_attention<128>(maps, a, grid, split, s);
  return launch_attention<64>(maps, a, grid, split, s);
}

}  // extern "C"
