// kda_selective.cu -- selective state space scan, for prompts and for single
// tokens.
//
//   dt = softplus(delta + delta_bias),  h[c,n] = exp(dt A[c,n]) h[c,n] + dt u[c] B[n]
//   y[c] = (sum_n C[n] h[c,n] + Dskip[c] u[c]) silu(z[c])
//
// exp(dt A) is taken as 2^(dt A log2 e), with A log2 e formed once per call in
// float32: its rounding is a relative change of A by at most 2^-24, so the
// state it decays is off by a like amount whatever the sequence's length.
#include <stdint.h>

#include "kda_launch.cuh"

namespace kda {
namespace {

constexpr int kScanThreads = 128;
constexpr int kPer = 4;  // state entries per thread
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float silu(float x) { return x / (1.f + expf(-x)); }

struct Rows {  // a strided input: batch and token stride in elements
  const void *p;
  long long sb, st;
};

struct ScanArgs {
  Rows u, delta, Bm, Cm, z;
  const float *A, *Dskip, *bias, *h0;
  const int *lens;
  void *y;
  float *hT;
  int B, T, D, G, softplus;
};

// One group of N / 4 lanes per (batch row, channel), token after token.
template <typename TI, int N>
__global__ void __launch_bounds__(kScanThreads) selective_scan_kernel(ScanArgs a) {
  constexpr int L = N / kPer;
  const long long id = (long long)blockIdx.x * (kScanThreads / L) + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  const bool live = id < (long long)a.B * a.D;
  const int b = live ? (int)(id / a.D) : 0, c = live ? (int)(id % a.D) : 0;
  const int g = c / (a.D / a.G);
  const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  const TI *u = static_cast<const TI *>(a.u.p) + b * a.u.sb + c;
  const TI *de = static_cast<const TI *>(a.delta.p) + b * a.delta.sb + c;
  const TI *Bm = static_cast<const TI *>(a.Bm.p) + b * a.Bm.sb + (long long)g * N + lane * kPer;
  const TI *Cm = static_cast<const TI *>(a.Cm.p) + b * a.Cm.sb + (long long)g * N + lane * kPer;
  const TI *z = static_cast<const TI *>(a.z.p);
  if (z) z += b * a.z.sb + c;
  const long long so = ((long long)b * a.D + c) * N + lane * kPer;
  const float bias = a.bias ? a.bias[c] : 0.f, skip = a.Dskip ? a.Dskip[c] : 0.f;
  float A2[kPer], h[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    A2[k] = a.A[(long long)c * N + lane * kPer + k] * kLog2e;
    h[k] = a.h0 ? a.h0[so + k] : 0.f;
  }
  // the lanes of a group share b, hence the trip count; a warp's groups may not
  for (int t = 0; t < len; ++t) {
    const float ut = Io<TI>::ld(u + t * a.u.st);
    float dt = Io<TI>::ld(de + t * a.delta.st) + bias;
    if (a.softplus) dt = softplus(dt);
    const float x = dt * ut;
    float acc = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      h[k] = exp2f(dt * A2[k]) * h[k] + x * Io<TI>::ld(Bm + t * a.Bm.st + k);
      acc += h[k] * Io<TI>::ld(Cm + t * a.Cm.st + k);
    }
    const unsigned mask = ((L == 32 ? 0u : (1u << (L & 31))) - 1u) << (threadIdx.x % 32 / L * L);
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(mask, acc, off);
    if (live && lane == 0) {
      acc += skip * ut;
      if (z) acc *= silu(Io<TI>::ld(z + t * a.z.st));
      Io<TI>::st(static_cast<TI *>(a.y) + ((long long)b * a.T + t) * a.D + c, acc);
    }
  }
  if (live && a.hT) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) a.hT[so + k] = h[k];
  }
}

struct StepArgs {
  Rows u, delta, Bm, Cm, z;  // st unused
  const float *A, *Dskip, *bias;
  float *S;
  const int *slots;
  int n_slots;
  void *y;
  int R, D, G, softplus;
};

template <typename TI, int N>
__global__ void __launch_bounds__(kScanThreads) selective_step_kernel(StepArgs a) {
  constexpr int L = N / kPer;
  const long long id = (long long)blockIdx.x * (kScanThreads / L) + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  if (id >= (long long)a.R * a.D) return;  // a whole group leaves at once
  const int r = (int)(id / a.D), c = (int)(id % a.D);
  const int slot = a.slots ? a.slots[r] : r;
  if (slot < 0 || slot >= a.n_slots) return;
  const int g = c / (a.D / a.G);
  float *S = a.S + ((long long)slot * a.D + c) * N + lane * kPer;
  const float ut = Io<TI>::ld(static_cast<const TI *>(a.u.p) + r * a.u.sb + c);
  float dt = Io<TI>::ld(static_cast<const TI *>(a.delta.p) + r * a.delta.sb + c) +
             (a.bias ? a.bias[c] : 0.f);
  if (a.softplus) dt = softplus(dt);
  const TI *Bm = static_cast<const TI *>(a.Bm.p) + r * a.Bm.sb + (long long)g * N + lane * kPer;
  const TI *Cm = static_cast<const TI *>(a.Cm.p) + r * a.Cm.sb + (long long)g * N + lane * kPer;
  float acc = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const float A2 = a.A[(long long)c * N + lane * kPer + k] * kLog2e;
    const float h = exp2f(dt * A2) * S[k] + dt * ut * Io<TI>::ld(Bm + k);
    S[k] = h;
    acc += h * Io<TI>::ld(Cm + k);
  }
  const unsigned mask = ((L == 32 ? 0u : (1u << (L & 31))) - 1u) << (threadIdx.x % 32 / L * L);
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(mask, acc, off);
  if (lane == 0) {
    if (a.Dskip) acc += a.Dskip[c] * ut;
    if (a.z.p) acc *= silu(Io<TI>::ld(static_cast<const TI *>(a.z.p) + r * a.z.sb + c));
    Io<TI>::st(static_cast<TI *>(a.y) + id, acc);
  }
}

template <typename TI, int N>
kda_status launch_scan(const ScanArgs &a, cudaStream_t st) {
  const long long per = kScanThreads / (N / kPer);
  const long long blocks = ((long long)a.B * a.D + per - 1) / per;
  if (blocks > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  selective_scan_kernel<TI, N><<<(unsigned)blocks, kScanThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
template <typename TI, int N>
kda_status launch_step(const StepArgs &a, cudaStream_t st) {
  const long long per = kScanThreads / (N / kPer);
  const long long blocks = ((long long)a.R * a.D + per - 1) / per;
  if (blocks > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  selective_step_kernel<TI, N><<<(unsigned)blocks, kScanThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename TI>
kda_status launch_scan_n(const ScanArgs &a, int N, cudaStream_t st) {
  switch (N) {
    case 8: return launch_scan<TI, 8>(a, st);
    case 16: return launch_scan<TI, 16>(a, st);
    case 32: return launch_scan<TI, 32>(a, st);
    default: return launch_scan<TI, 64>(a, st);
  }
}
template <typename TI>
kda_status launch_step_n(const StepArgs &a, int N, cudaStream_t st) {
  switch (N) {
    case 8: return launch_step<TI, 8>(a, st);
    case 16: return launch_step<TI, 16>(a, st);
    case 32: return launch_step<TI, 32>(a, st);
    default: return launch_step<TI, 64>(a, st);
  }
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t size_of(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }

// Checks shared by the scan and the step: enums, flags, sizes.
kda_status check_sizes(int B, int T, int D, int G, int N, kda_dtype dt, unsigned flags) {
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if ((flags & ~KDA_SCAN_SOFTPLUS) != 0u) return KDA_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || D < 1 || G < 1 || D % G != 0) return KDA_ERR_INVALID_ARG;
  if (N != 8 && N != 16 && N != 32 && N != 64) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace
}  // namespace kda

extern "C" size_t kda_selective_scan_workspace_size(int B, int T, int D, int G, int N,
                                                    kda_dtype dt) {
  return kda::check_sizes(B, T, D, G, N, dt, 0u) == KDA_OK ? 256 : 0;
}

extern "C" kda_status kda_selective_scan(const void *u, const void *delta, const float *A,
                                         const void *Bm, const void *Cm, const float *Dskip,
                                         const void *z, const float *delta_bias, const float *h0,
                                         const int *lens, void *y, float *hT,
                                         const long long *strides, int B, int T, int D, int G,
                                         int N, kda_dtype dt, unsigned flags, void *workspace,
                                         size_t workspace_bytes, kda_stream_t stream) {
  using namespace kda;
  const kda_status ok = check_sizes(B, T, D, G, N, dt, flags);
  if (ok != KDA_OK) return ok;
  if (B == 0 || (T == 0 && !hT)) return KDA_OK;
  if (!A || !strides || (T > 0 && (!u || !delta || !Bm || !Cm || !y))) return KDA_ERR_INVALID_ARG;
  for (int i = 0; i < (z ? 10 : 8); ++i)
    if (strides[i] < 0) return KDA_ERR_INVALID_ARG;
  const uintptr_t e = size_of(dt);
  if (!aligned(u, e) || !aligned(delta, e) || !aligned(Bm, e) || !aligned(Cm, e) ||
      !aligned(z, e) || !aligned(A, 16) || !aligned(Dskip, 16) || !aligned(delta_bias, 16) ||
      !aligned(h0, 16) || !aligned(lens, 4) || !aligned(y, 16) || !aligned(hT, 16))
    return KDA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < kda_selective_scan_workspace_size(B, T, D, G, N, dt))
    return KDA_ERR_INVALID_ARG;
  const ScanArgs a{{u, strides[0], strides[1]},
                   {delta, strides[2], strides[3]},
                   {Bm, strides[4], strides[5]},
                   {Cm, strides[6], strides[7]},
                   {z, z ? strides[8] : 0, z ? strides[9] : 0},
                   A, Dskip, delta_bias, h0, lens, y, hT, B, T, D, G,
                   (flags & KDA_SCAN_SOFTPLUS) != 0u};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dt == KDA_BF16 ? launch_scan_n<__nv_bfloat16>(a, N, st) : launch_scan_n<float>(a, N, st);
}

extern "C" kda_status kda_selective_step(const void *u, const void *delta, const float *A,
                                         const void *Bm, const void *Cm, const float *Dskip,
                                         const void *z, const float *delta_bias, float *S,
                                         const int *slots, int n_slots, void *y,
                                         const long long *strides, int R, int D, int G, int N,
                                         kda_dtype dt, unsigned flags, kda_stream_t stream) {
  using namespace kda;
  const kda_status ok = check_sizes(R, 1, D, G, N, dt, flags);
  if (ok != KDA_OK) return ok;
  if (n_slots < 0 || (!slots && R > n_slots)) return KDA_ERR_INVALID_ARG;
  if (R == 0 || n_slots == 0) return KDA_OK;
  if (!u || !delta || !A || !Bm || !Cm || !S || !y || !strides) return KDA_ERR_INVALID_ARG;
  for (int i = 0; i < (z ? 5 : 4); ++i)
    if (strides[i] < 0) return KDA_ERR_INVALID_ARG;
  const uintptr_t e = size_of(dt);
  if (!aligned(u, e) || !aligned(delta, e) || !aligned(Bm, e) || !aligned(Cm, e) ||
      !aligned(z, e) || !aligned(A, 16) || !aligned(Dskip, 16) || !aligned(delta_bias, 16) ||
      !aligned(S, 16) || !aligned(slots, 4) || !aligned(y, 16))
    return KDA_ERR_INVALID_ARG;
  const StepArgs a{{u, strides[0], 0}, {delta, strides[1], 0}, {Bm, strides[2], 0},
                   {Cm, strides[3], 0}, {z, z ? strides[4] : 0, 0},
                   A, Dskip, delta_bias, S, slots, n_slots, y, R, D, G,
                   (flags & KDA_SCAN_SOFTPLUS) != 0u};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dt == KDA_BF16 ? launch_step_n<__nv_bfloat16>(a, N, st) : launch_step_n<float>(a, N, st);
}
