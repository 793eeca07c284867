// Entry point of the few-row linear on NVFP4 weights.  Included at the end of nvfp4_api.cu, whose helpers
// (argument checks, per-device state) it uses.
#pragma once

#include "w4a16.cuh"

namespace {

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

// Rows that the kernels are built for: the digits of 2, 8, 16 or 32 rows are 16, 48, 96 or 192 columns.
int w4_rows(int64_t M) { return M <= 2 ? 2 : M <= 8 ? 8 : M <= 16 ? 16 : 32; }

// Workspace: chunk images, 32 row factors, partial sums per (unit + CTA).
struct W4Space {
  size_t images, factors, partials;
  size_t total() const { return images + factors + partials; }
};

W4Space w4_space(int64_t M, int64_t N, int64_t K) {
  const int mp = w4_rows(M);
  const size_t units = static_cast<size_t>((N + 255) / 256);
  W4Space s;
  s.images = static_cast<size_t>((K + kW4Chunk - 1) / kW4Chunk) * w4_image_bytes(mp);
  s.factors = 128;
  s.partials = (units + kW4MaxCtas) * 2 * mp * 128 * 4;
  return s;
}

// A launch that may start while the one before in the stream runs (its kernel waits for that one's end itself).
template <typename... Params, typename... Args>
cudaError_t w4_launch(void (*kernel)(Params...), int grid, int block, size_t smem, int cluster, bool early, cudaStream_t s,
                      const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (early) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = static_cast<unsigned>(n);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int MP, bool kFused>
nvfp4_status launch_w4a16(DeviceState* st, const CUtensorMap& map, const W4Args& a, int ctas, cudaStream_t s) {
  using C = W4Cfg<MP, kFused>;
  auto kernel = w4a16_kernel<MP, kFused>;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    bool& attr = st->smem_attr_set_w4[kFused ? 4 : MP == 2 ? 0 : 1 + MP / 16];
    if (!attr) {
      // the other kernels run with this one's split of L1 and shared memory: an SM changes it only when idle, so
      // this one could not start beside them (32 rows of K = 53248: 12 us later)
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess ||
          (!kFused && cudaFuncSetAttribute(w4a16_prepare_kernel<MP>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                           cudaSharedmemCarveoutMaxShared) != cudaSuccess) ||
          cudaFuncSetAttribute(w4a16_finish_kernel<MP>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return NVFP4_ERR_CUDA;
      attr = true;
    }
  }
  cudaError_t err = cudaSuccess;
  if (!kFused) {
    // enough CTAs per row for 4 elements per thread, at most a cluster of 8 and two CTAs per SM
    const int per_row = std::max(1, std::min({8, 2 * st->sm_count / a.M, (a.K / 4 + kW4PrepThreads - 1) / kW4PrepThreads}));
    err = w4_launch(w4a16_prepare_kernel<MP>, a.M * per_row, kW4PrepThreads, 0, per_row, false, s, a);
  }
  if (err == cudaSuccess) err = w4_launch(kernel, ctas, kW4Threads, C::SMEM_BYTES, 1, !kFused, s, map, a);
  const int tasks = a.units * (a.kind == NVFP4_EPI_GATED_SILU ? 1 : 2) * a.M;
  if (err == cudaSuccess) err = w4_launch(w4a16_finish_kernel<MP>, (tasks + 3) / 4, 128, 0, 1, true, s, a);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

extern "C" {

size_t nvfp4_w4a16_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t most = int64_t(1) << 30;
  if (M < 1 || M > kW4MaxRows || N < 1 || N > most || K < 1 || K > most) return 0;
  return w4_space(M, N, K).total();
}

nvfp4_status nvfp4_w4a16_linear(const void* x, int64_t M, int64_t ldx, int32_t silu_input, const nvfp4_tensor* w,
                                const nvfp4_epilogue_desc* epi, void* out, int64_t ld_out, void* workspace,
                                size_t workspace_bytes, nvfp4_stream_t stream) {
  if (!epi || M < 0) return NVFP4_ERR_INVALID_ARG;
  if (nvfp4_status e = check_tensor(w, true, 16)) return e;
  const int64_t N = w->rows, K = w->cols;
  if (N < 1) return NVFP4_ERR_INVALID_ARG;
  if (epi->kind != NVFP4_EPI_BIAS && epi->kind != NVFP4_EPI_GATED_SILU && epi->kind != NVFP4_EPI_RESID_GATE)
    return NVFP4_ERR_INVALID_ARG;
  if (epi->out_nvfp4 || epi->out_amax) return NVFP4_ERR_INVALID_ARG;
  const bool gated = epi->kind == NVFP4_EPI_GATED_SILU;
  if (M > kW4MaxRows || K % 64 || N > (int64_t(1) << 30) || K > (int64_t(1) << 30) || (gated && N % 256))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return NVFP4_OK;
  const int64_t n_out = gated ? N / 2 : N;
  if (!x || !out || !workspace || ldx < K || ld_out < n_out) return NVFP4_ERR_INVALID_ARG;
  if (epi->kind == NVFP4_EPI_RESID_GATE && (!epi->residual || !epi->gate || epi->ld_residual < n_out))
    return NVFP4_ERR_INVALID_ARG;
  if (workspace_bytes < w4_space(M, N, K).total()) return NVFP4_ERR_SCRATCH_LIMIT;
  if (!aligned16(workspace) || !aligned16(x) || (ldx * 2) % 16 || !aligned2(out) || !aligned2(epi->bias) ||
      (epi->kind == NVFP4_EPI_RESID_GATE && (!aligned2(epi->residual) || !aligned4(epi->gate))))
    return NVFP4_ERR_MISALIGNED;
  DeviceState* st;
  if (nvfp4_status e = device_state(&st)) return e;
  W4Args a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.ldx = ldx;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.silu = silu_input != 0;
  a.scales = static_cast<const uint8_t*>(w->scales);
  a.k_atoms = static_cast<int>(k_atoms_of(K));
  a.g = w->tensor_scale;
  a.chunks = static_cast<int>((K + kW4Chunk - 1) / kW4Chunk);
  a.units = static_cast<int>(gated ? N / 256 : (N + 255) / 256);
  const int64_t line = static_cast<int64_t>(a.units) * a.chunks;
  if (line > kW4MaxLine) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int ctas = static_cast<int>(std::min<int64_t>(std::min(st->sm_count, kW4MaxCtas), line));
  a.base = static_cast<int>(line / ctas);
  a.rest = static_cast<int>(line % ctas);
  const W4Space space = w4_space(M, N, K);
  a.digits = static_cast<uint8_t*>(workspace);
  a.factor = reinterpret_cast<float*>(a.digits + space.images);
  a.partial = reinterpret_cast<float*>(a.digits + space.images + space.factors);
  a.bias = static_cast<const __nv_bfloat16*>(epi->bias);
  a.residual = static_cast<const __nv_bfloat16*>(epi->residual);
  a.ld_res = epi->ld_residual;
  a.gate = epi->gate;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.ld_out = ld_out;
  a.kind = epi->kind;
  a.error_word = st->error_word;
  a.timeout_ns = wait_timeout_ns();
#ifdef NVFP4_TEST_HOOKS
  a.test_withhold = g_test_withhold_arrivals.load();
#endif
  CUtensorMap map;
  if (nvfp4_status e = make_code_map(&map, w)) return e;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // One or two rows: a CTA makes the digits of the chunks in its range for itself, if that is less work than another launch.
  // Weights that are not in L2, own digits against a kernel's.  One row: [4608 x 256] (1 chunk) 5.0 and 5.6 us, [4608 x 4608]
  // (3) 7.9 and 9.3, [27648 x 4608] (14) 17.2 and 19.2, [32768 x 4608] (16) 19.6 and 21.5, [4608 x 29952] (15) 20.2 and 20.7.
  // Two rows: [13824 x 4608] (7) 12.9 and 13.8, [4608 x 13824] (7) 14.4 and 14.4, [4608 x 18432] (9) 16.4 and 15.5, [27648 x
  // 4608] (14) 19.7 and 19.4.
  const bool fused = M <= kW4FusedRows && M * std::min<int64_t>(a.chunks, a.base + 1) <= kW4FusedChunks;
  switch (w4_rows(M)) {
    case 2:
      return fused ? launch_w4a16<2, true>(st, map, a, ctas, s) : launch_w4a16<2, false>(st, map, a, ctas, s);
    case 8: return launch_w4a16<8, false>(st, map, a, ctas, s);
    case 16: return launch_w4a16<16, false>(st, map, a, ctas, s);
    default: return launch_w4a16<32, false>(st, map, a, ctas, s);
  }
}

}  // extern "C"
