// kv8_cache.cu -- the rolling token cache in 8 bits: runs of tokens quantised as
// they are written (swa_kv8_write) and read back (swa_kv8_read).  The format is
// kv8.cuh's.
//
// Bound: device memory.  A row of D elements belongs to D / 8 neighbouring lanes,
// eight elements each (16 bytes in, 8 out at 16 bits), whose largest magnitude is a
// few shuffles; nothing is kept between rows.  The cache's slots are the rolling
// ones, position mod W, so a run may wrap around its end.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/swa.h"
#include "internal.h"
#include "kv8.cuh"

namespace swa {
namespace {

constexpr int kRunThreads = 256;

struct RunParams {
  void* x[2];             // K and V rows [B, T, Hkv, D]
  uint8_t* x8[2];         // [B, W, Hkv, D]
  uint8_t* exp[2];        // [B, Hkv, W]
  const long long* pos;   // [B]
  const int* count;       // [B] or null
  int B, T, W, Hkv;
};

SWA_DEV int run_length(const RunParams& p, int b) {
  return p.count ? min(max(p.count[b], 0), p.T) : p.T;
}

// grid: x over rows of one sequence (token, head), y the sequence, z K or V
template <typename T, int D>
__global__ void __launch_bounds__(kRunThreads) kv8_write_kernel(const __grid_constant__ RunParams p) {
  constexpr int kLanes = D / 8;
  const int b = blockIdx.y, kv = blockIdx.z;
  const long long pos = p.pos[b];
  const int n = run_length(p, b);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kRunThreads / kLanes) + threadIdx.x / kLanes;
  const int t = static_cast<int>(r / p.Hkv), h = static_cast<int>(r - static_cast<int64_t>(t) * p.Hkv);
  const int part = threadIdx.x % kLanes;
  // of a run longer than the window only the last W tokens stay
  const bool live = pos >= 0 && t < n && t >= n - p.W;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live)
    load8(static_cast<const T*>(p.x[kv]) + ((static_cast<int64_t>(b) * p.T + t) * p.Hkv + h) * D + part * 8, v);
  float a = amax8(v);
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  if (!live) return;
  const int e = kv8_exponent(a);
  const int64_t slot = (pos + t) % p.W;
  *reinterpret_cast<uint2*>(p.x8[kv] + ((static_cast<int64_t>(b) * p.W + slot) * p.Hkv + h) * D + part * 8) =
      quantise8(v, e);
  if (part == 0)
    p.exp[kv][(static_cast<int64_t>(b) * p.Hkv + h) * p.W + slot] = static_cast<uint8_t>(e + 127);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRunThreads) kv8_read_kernel(const __grid_constant__ RunParams p) {
  constexpr int kLanes = D / 8;
  const int b = blockIdx.y, kv = blockIdx.z;
  const long long pos = p.pos[b];
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kRunThreads / kLanes) + threadIdx.x / kLanes;
  const int t = static_cast<int>(r / p.Hkv), h = static_cast<int>(r - static_cast<int64_t>(t) * p.Hkv);
  const int part = threadIdx.x % kLanes;
  if (pos < 0 || t >= run_length(p, b)) return;
  const int64_t slot = (pos + t) % p.W;
  const uint2 q = *reinterpret_cast<const uint2*>(
      p.x8[kv] + ((static_cast<int64_t>(b) * p.W + slot) * p.Hkv + h) * D + part * 8);
  float v[8];
  dequantise8(q, p.exp[kv][(static_cast<int64_t>(b) * p.Hkv + h) * p.W + slot] - 127, v);
  store8(static_cast<T*>(p.x[kv]) + ((static_cast<int64_t>(b) * p.T + t) * p.Hkv + h) * D + part * 8, v);
}

template <bool kWrite, typename T, int D>
cudaError_t launch_run(const RunParams& p, cudaStream_t st) {
  constexpr int kRows = kRunThreads / (D / 8);
  const int64_t rows = static_cast<int64_t>(p.T) * p.Hkv;
  const dim3 grid(static_cast<unsigned>((rows + kRows - 1) / kRows), p.B, 2);
  if (kWrite)
    kv8_write_kernel<T, D><<<grid, kRunThreads, 0, st>>>(p);
  else
    kv8_read_kernel<T, D><<<grid, kRunThreads, 0, st>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

template <bool kWrite, typename T>
cudaError_t launch_run_d(const RunParams& p, int D, cudaStream_t st) {
  if (D == 32) return launch_run<kWrite, T, 32>(p, st);
  if (D == 64) return launch_run<kWrite, T, 64>(p, st);
  return launch_run<kWrite, T, 128>(p, st);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool kWrite>
swa_status run(void* k, void* v, void* k8, uint8_t* k_exp, void* v8, uint8_t* v_exp, const long long* pos,
               const int32_t* count, int B, int T, int W, int Hkv, int D, int dtype, void* stream) {
  if (B < 0 || T < 0 || W < 1 || Hkv < 1 || D < 1) return SWA_ERR_ARG;
  if (dtype != SWA_F32 && dtype != SWA_BF16) return SWA_ERR_ARG;
  if (D != 32 && D != 64 && D != 128) return SWA_ERR_UNSUPPORTED;
  if (B > 65535 || static_cast<int64_t>(T) * Hkv > (1ll << 33)) return SWA_ERR_SHAPE;
  if (B == 0 || T == 0) return SWA_OK;
  if (!k || !v || !k8 || !k_exp || !v8 || !v_exp || !pos) return SWA_ERR_ARG;
  if (!al16(k) || !al16(v) || !al16(k8) || !al16(v8) || (reinterpret_cast<uintptr_t>(pos) & 7u) ||
      (reinterpret_cast<uintptr_t>(count) & 3u))
    return SWA_ERR_ARG;
  int* err = nullptr;
  if (const int ds = device_ready_status(&err)) return static_cast<swa_status>(ds);
  RunParams p{{k, v}, {static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8)}, {k_exp, v_exp}, pos, count, B, T, W, Hkv};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SWA_BF16 ? launch_run_d<kWrite, __nv_bfloat16>(p, D, st)
                                          : launch_run_d<kWrite, float>(p, D, st);
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

}  // namespace
}  // namespace swa

extern "C" swa_status swa_kv8_write(const void* k, const void* v, void* k8, uint8_t* k_exp, void* v8,
                                    uint8_t* v_exp, const long long* pos, const int32_t* count, int B, int T, int W,
                                    int Hkv, int head_dim, int dtype, void* stream) {
  return swa::run<true>(const_cast<void*>(k), const_cast<void*>(v), k8, k_exp, v8, v_exp, pos, count, B, T, W, Hkv,
                        head_dim, dtype, stream);
}

extern "C" swa_status swa_kv8_read(const void* k8, const uint8_t* k_exp, const void* v8, const uint8_t* v_exp,
                                   const long long* pos, const int32_t* count, void* k, void* v, int B, int T, int W,
                                   int Hkv, int head_dim, int dtype, void* stream) {
  return swa::run<false>(k, v, const_cast<void*>(k8), const_cast<uint8_t*>(k_exp), const_cast<void*>(v8),
                         const_cast<uint8_t*>(v_exp), pos, count, B, T, W, Hkv, head_dim, dtype, stream);
}
