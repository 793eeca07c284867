// Entry point of the head norm with position rotation.  Included at the end of nvfp4_api.cu, whose
// helpers (argument checks, per-device state) it uses.
#pragma once

#include "norm_rope.cuh"

namespace {

// x and out of an empty call may be NULL.
nvfp4_status check_heads(const nvfp4_heads* h, int64_t rows, int32_t head_dim, float eps) {
  if ((rows > 0 && (!h->x || !h->out)) || h->heads <= 0) return NVFP4_ERR_INVALID_ARG;
  if (h->heads > 1 && (h->head_stride < head_dim || h->out_head_stride < head_dim)) return NVFP4_ERR_INVALID_ARG;
  if (rows > 1 && (h->row_stride < 0 || h->out_row_stride < head_dim)) return NVFP4_ERR_INVALID_ARG;
  if (h->heads > 65535) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (h->gamma && !(eps > 0.0f && eps < 3.0e38f)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(h->x) || !aligned16(h->out) || (rows > 1 && (h->row_stride % 8 || h->out_row_stride % 8)) ||
      (h->heads > 1 && (h->head_stride % 8 || h->out_head_stride % 8)) || (h->gamma && !aligned16(h->gamma)))
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

RopeHeads rope_heads(const nvfp4_heads* h, int32_t head_dim, int steps) {
  RopeHeads r{};
  if (!h) return r;
  r.x = static_cast<const __nv_bfloat16*>(h->x);
  r.out = static_cast<__nv_bfloat16*>(h->out);
  r.row = h->row_stride;
  r.head = h->head_stride;
  r.out_row = h->out_row_stride;
  r.out_head = h->out_head_stride;
  r.gamma = static_cast<const __nv_bfloat16*>(h->gamma);
  r.heads = h->heads;
  const int per_chunk = steps * (256 / head_dim);
  r.chunks = (h->heads + per_chunk - 1) / per_chunk;
  return r;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_qk_norm_rope(const nvfp4_heads* q, const nvfp4_heads* k, int64_t rows, int32_t head_dim,
                                const nvfp4_rope_desc* rope, nvfp4_stream_t stream) {
  if (!q || !rope || rows < 0) return NVFP4_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (nvfp4_status e = check_heads(q, rows, head_dim, rope->eps)) return e;
  if (k)
    if (nvfp4_status e = check_heads(k, rows, head_dim, rope->eps)) return e;
  if (rope->rot_dim < 0 || rope->rot_dim > head_dim || rope->rot_dim % 16) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (rope->rot_dim > 0) {
    if (!rope->cos || !rope->sin || rope->table_rows <= 0 || rope->ld_table < rope->rot_dim / 2)
      return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(rope->cos) || !aligned16(rope->sin) || rope->ld_table % 4 ||
        (rope->positions && !aligned4(rope->positions)))
      return NVFP4_ERR_MISALIGNED;
  }
  if (rows == 0) return NVFP4_OK;
  // A warp has kRopeFlight steps of a row's heads, or, from 24 rows per SM on, all of them, which saves the reads of tables and
  // gamma.  18 heads of 256 for q and k, inputs larger than L2 in all, steps against all heads.  Pairs of halves: 37 rows 3.3
  // and 6.5 us, 2400 rows 20.4 and 21.3, 2816 rows 23.8 and 23.5, 3552 rows 28.4 and 25.5, 4608 rows 35.2 and 33.5, 16896 rows
  // 115 and 105.  Neighbours: 37 rows 3.1 and 6.2, 2400 rows 18.2 and 20.8, and within 3% either way from 3552 rows on.
  const RopeHeads few_q = rope_heads(q, head_dim, kRopeFlight), few_k = rope_heads(k, head_dim, kRopeFlight);
  if (rows > (int64_t(1) << 31) / (static_cast<int64_t>(few_q.chunks) + few_k.chunks)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  DeviceState* st;
  if (nvfp4_status e = device_state(&st)) return e;
  const int most_heads = std::max(q->heads, k ? k->heads : 0), per_step = 256 / head_dim;
  int steps = kRopeFlight;
  if (rows >= 24 * st->sm_count) steps = (most_heads + per_step - 1) / per_step;
  RopeArgs a{};
  a.q = rope_heads(q, head_dim, steps);
  a.k = rope_heads(k, head_dim, steps);
  a.steps = steps;
  a.rows = rows;
  a.rot = rope->rot_dim;
  a.eps = rope->eps;
  a.table_rows = 1;
  if (a.rot > 0) {
    a.cos = rope->cos;
    a.sin = rope->sin;
    a.table_rows = rope->table_rows;
    a.ld_table = rope->ld_table;
    a.positions = rope->positions;
  }
  // one warp per (row, chunk of heads); the unit number is 32 bits in the kernel
  const int64_t chunks = static_cast<int64_t>(a.q.chunks) + a.k.chunks;
  const int grid = static_cast<int>((rows * chunks + 7) / 8);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool il = rope->interleaved != 0;
  auto kernel = head_dim == 256 ? (il ? qk_norm_rope_kernel<256, true> : qk_norm_rope_kernel<256, false>)
                : head_dim == 128 ? (il ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>)
                                  : (il ? qk_norm_rope_kernel<64, true> : qk_norm_rope_kernel<64, false>);
  kernel<<<grid, 256, 0, s>>>(a);
  return launch_status();
}

}  // extern "C"
