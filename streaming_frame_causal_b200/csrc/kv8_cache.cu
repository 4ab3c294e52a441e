// kv8_cache.cu -- the rolling token cache in 8 bits: runs of tokens quantised as
// they are written (swa_kv8_write) and read back (swa_kv8_read).  The format is
// kv8.cuh's.
//
// Bound: device memory.  A row of D elements belongs to D / 16 neighbouring lanes,
// 16 elements each (16 bytes of the cache), whose largest magnitude is a few
// shuffles; a thread loads its part of kRunRows rows before it works on the
// first.  The cache's slots are the rolling ones, position mod W, so a run may wrap
// around its end.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/swa.h"
#include "fastdiv.cuh"
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
  FastDiv heads;          // Hkv
};

SWA_DEV int run_length(const RunParams& p, int b) {
  return p.count ? min(max(p.count[b], 0), p.T) : p.T;
}

constexpr int kRunRows = 4;  // rows of a thread

// 16 elements as they are stored
template <typename T>
struct Raw16 {
  static constexpr int kWords = sizeof(T);
  uint4 w[kWords];
  SWA_DEV void load(const T* x) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(x)[i];
  }
  SWA_DEV void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  SWA_DEV void widen(float* v) const {
    const T* x = reinterpret_cast<const T*>(w);
    load8(x, v);
    load8(x + 8, v + 8);
  }
};

// The rows (token, head) of a thread in one sequence's run: r0, r0 + step, ...
template <int D>
struct RunRows {
  static constexpr int kLanes = D / 16;
  static constexpr int kStep = kRunThreads / kLanes;
  int r0, part;
  SWA_DEV RunRows()
      : r0(static_cast<int>(blockIdx.x) * (kStep * kRunRows) + threadIdx.x / kLanes), part(threadIdx.x % kLanes) {}
};

// grid: x over the rows of one sequence, y the sequence, z K or V
template <typename T, int D>
__global__ void __launch_bounds__(kRunThreads) kv8_write_kernel(const __grid_constant__ RunParams p) {
  using R = RunRows<D>;
  const R at;
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z;
  const long long pos = p.pos[b];
  // of a run longer than the window only the last W tokens stay
  const int end = run_length(p, b) * p.Hkv, skip = max(0, run_length(p, b) - p.W);
  if (pos < 0 || at.r0 - static_cast<int>(threadIdx.x) / R::kLanes >= end) return;
  const T* x = static_cast<const T*>(is_v ? p.x[1] : p.x[0]) + static_cast<int64_t>(b) * p.T * p.Hkv * D + at.part * 16;
  Raw16<T> raw[kRunRows];
  bool live[kRunRows];
#pragma unroll
  for (int i = 0; i < kRunRows; ++i) {
    const int r = at.r0 + i * R::kStep;
    live[i] = r < end && r >= skip * p.Hkv;
    if (live[i]) raw[i].load(x + static_cast<int64_t>(r) * D);
    else raw[i].clear();
  }
  uint8_t* x8 = (is_v ? p.x8[1] : p.x8[0]) + static_cast<int64_t>(b) * p.W * p.Hkv * D + at.part * 16;
  uint8_t* exps = (is_v ? p.exp[1] : p.exp[0]) + static_cast<int64_t>(b) * p.Hkv * p.W;
  const int slot0 = static_cast<int>((pos + skip) % p.W);
#pragma unroll
  for (int i = 0; i < kRunRows; ++i) {
    float v[16];
    raw[i].widen(v);
    float a = fmaxf(amax8(v), amax8(v + 8));
#pragma unroll
    for (int off = R::kLanes / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    if (live[i]) {
      int h;
      const int t = p.heads.divmod(at.r0 + i * R::kStep, h) - skip;  // < W
      const int64_t slot = t < p.W - slot0 ? slot0 + t : t - (p.W - slot0);
      const int e = kv8_exponent(a);
      const uint2 lo = quantise8(v, e), hi = quantise8(v + 8, e);
      *reinterpret_cast<uint4*>(x8 + (slot * p.Hkv + h) * D) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      if (at.part == 0) exps[h * static_cast<int64_t>(p.W) + slot] = static_cast<uint8_t>(e + 127);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kRunThreads) kv8_read_kernel(const __grid_constant__ RunParams p) {
  using R = RunRows<D>;
  const R at;
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z;
  const long long pos = p.pos[b];
  const int rows = run_length(p, b) * p.Hkv;
  if (pos < 0 || at.r0 >= rows) return;
  const uint8_t* x8 = (is_v ? p.x8[1] : p.x8[0]) + static_cast<int64_t>(b) * p.W * p.Hkv * D + at.part * 16;
  const uint8_t* exps = (is_v ? p.exp[1] : p.exp[0]) + static_cast<int64_t>(b) * p.Hkv * p.W;
  const int slot0 = static_cast<int>(pos % p.W);
  uint4 q[kRunRows];
  int e[kRunRows];
#pragma unroll
  for (int i = 0; i < kRunRows; ++i) {
    const int r = at.r0 + i * R::kStep;
    if (r < rows) {
      int h;
      int64_t slot = slot0 + static_cast<int64_t>(p.heads.divmod(r, h));
      if (slot >= p.W) slot %= p.W;
      q[i] = *reinterpret_cast<const uint4*>(x8 + (slot * p.Hkv + h) * D);
      e[i] = exps[h * static_cast<int64_t>(p.W) + slot] - 127;
    }
  }
  T* x = static_cast<T*>(is_v ? p.x[1] : p.x[0]) + static_cast<int64_t>(b) * p.T * p.Hkv * D + at.part * 16;
#pragma unroll
  for (int i = 0; i < kRunRows; ++i) {
    const int r = at.r0 + i * R::kStep;
    if (r < rows) {
      T* y = x + static_cast<int64_t>(r) * D;
      float v[8];
      dequantise8(make_uint2(q[i].x, q[i].y), e[i], v);
      store8(y, v);
      dequantise8(make_uint2(q[i].z, q[i].w), e[i], v);
      store8(y + 8, v);
    }
  }
}

template <bool kWrite, typename T, int D>
cudaError_t launch_run(const RunParams& p, cudaStream_t st) {
  constexpr int kRows = RunRows<D>::kStep * kRunRows;
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
  if (B > 65535 || static_cast<int64_t>(T) * Hkv >= (1ll << 30)) return SWA_ERR_SHAPE;
  if (B == 0 || T == 0) return SWA_OK;
  if (!k || !v || !k8 || !k_exp || !v8 || !v_exp || !pos) return SWA_ERR_ARG;
  if (!al16(k) || !al16(v) || !al16(k8) || !al16(v8) || (reinterpret_cast<uintptr_t>(pos) & 7u) ||
      (reinterpret_cast<uintptr_t>(count) & 3u))
    return SWA_ERR_ARG;
  int* err = nullptr;
  if (const int ds = device_ready_status(&err)) return static_cast<swa_status>(ds);
  RunParams p{{k, v}, {static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8)}, {k_exp, v_exp}, pos, count, B, T, W, Hkv, FastDiv(Hkv)};
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
