// kda_short_conv.cu -- short causal convolution over time, for prompts and
// for single tokens.
//
//   y[t] = act(bias + sum_{j<W} w[j] xx[t + j]),   xx = [s0 ; x] along time,
//
// per channel of each head, with W in {2, 3, 4} taps and the last W - 1
// inputs handed on as the state.
#include <stdint.h>

#include "kda_launch.cuh"

namespace kda {
namespace {

constexpr int kConvThreads = 128;

__device__ __forceinline__ float conv_act(float v, int silu) {
  return silu ? v / (1.f + expf(-v)) : v;
}

struct ConvArgs {
  const void *x;
  long long x_sb, x_sh, x_st;
  const float *w, *bias;
  const void *s0;
  const int *lens;
  void *y, *sT;
  int B, H, T, d, silu;
};

// One thread per (batch row, channel), token after token.
template <typename TI, int W>
__global__ void __launch_bounds__(kConvThreads) short_conv_kernel(ConvArgs a) {
  const long long C = (long long)a.H * a.d;
  const long long id = (long long)blockIdx.x * kConvThreads + threadIdx.x;
  if (id >= C * a.B) return;
  const int b = (int)(id / C);
  const int h = (int)(id % C / a.d), i = (int)(id % a.d);
  const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
  const TI *x = static_cast<const TI *>(a.x) + b * a.x_sb + h * a.x_sh + i;
  TI *y = static_cast<TI *>(a.y) + ((long long)b * a.H + h) * a.T * a.d + i;
  const long long so = ((long long)b * a.H + h) * (W - 1) * a.d + i;
  float w[W], win[W];
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = a.w[((long long)h * a.d + i) * W + j];
  const float bias = a.bias ? a.bias[(long long)h * a.d + i] : 0.f;
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    win[j] = a.s0 ? Io<TI>::ld(static_cast<const TI *>(a.s0) + so + (long long)j * a.d) : 0.f;
  for (int t = 0; t < len; ++t) {
    win[W - 1] = Io<TI>::ld(x + t * a.x_st);
    float v = bias;
#pragma unroll
    for (int j = 0; j < W; ++j) v += w[j] * win[j];
    Io<TI>::st(y + (long long)t * a.d, conv_act(v, a.silu));
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
  }
  if (a.sT) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      Io<TI>::st(static_cast<TI *>(a.sT) + so + (long long)j * a.d, win[j]);
  }
}

struct ConvStepArgs {
  const void *x;
  long long x_sn, x_sh;
  const float *w, *bias;
  void *S;
  const int *slots;
  int n_slots;
  void *y;
  int N, H, d, silu;
};

template <typename TI, int W>
__global__ void __launch_bounds__(kConvThreads) short_conv_step_kernel(ConvStepArgs a) {
  const long long C = (long long)a.H * a.d;
  const long long id = (long long)blockIdx.x * kConvThreads + threadIdx.x;
  if (id >= C * a.N) return;
  const int n = (int)(id / C);
  const int h = (int)(id % C / a.d), i = (int)(id % a.d);
  const int slot = a.slots ? a.slots[n] : n;
  if (slot < 0 || slot >= a.n_slots) return;
  TI *S = static_cast<TI *>(a.S) + ((long long)slot * a.H + h) * (W - 1) * a.d + i;
  const float *w = a.w + ((long long)h * a.d + i) * W;
  float v = a.bias ? a.bias[(long long)h * a.d + i] : 0.f;
  float win[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j] = Io<TI>::ld(S + (long long)j * a.d);
  win[W - 1] = Io<TI>::ld(static_cast<const TI *>(a.x) + n * a.x_sn + h * a.x_sh + i);
#pragma unroll
  for (int j = 0; j < W; ++j) v += w[j] * win[j];
  Io<TI>::st(static_cast<TI *>(a.y) + id, conv_act(v, a.silu));
#pragma unroll
  for (int j = 0; j < W - 1; ++j) Io<TI>::st(S + (long long)j * a.d, win[j + 1]);
}

template <typename TI>
kda_status launch_conv(const ConvArgs &a, int W, cudaStream_t st) {
  const long long blocks = ((long long)a.B * a.H * a.d + kConvThreads - 1) / kConvThreads;
  if (blocks > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  const unsigned g = (unsigned)blocks;
  if (W == 2) short_conv_kernel<TI, 2><<<g, kConvThreads, 0, st>>>(a);
  if (W == 3) short_conv_kernel<TI, 3><<<g, kConvThreads, 0, st>>>(a);
  if (W == 4) short_conv_kernel<TI, 4><<<g, kConvThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename TI>
kda_status launch_conv_step(const ConvStepArgs &a, int W, cudaStream_t st) {
  const long long blocks = ((long long)a.N * a.H * a.d + kConvThreads - 1) / kConvThreads;
  if (blocks > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  const unsigned g = (unsigned)blocks;
  if (W == 2) short_conv_step_kernel<TI, 2><<<g, kConvThreads, 0, st>>>(a);
  if (W == 3) short_conv_step_kernel<TI, 3><<<g, kConvThreads, 0, st>>>(a);
  if (W == 4) short_conv_step_kernel<TI, 4><<<g, kConvThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t size_of(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }

}  // namespace
}  // namespace kda

extern "C" kda_status kda_short_conv(const void *x, long long x_sb, long long x_sh, long long x_st,
                                     const float *w, const float *bias, const void *s0,
                                     const int *lens, void *y, void *sT, int B, int H, int T,
                                     int d, int W, kda_dtype dt, kda_act act,
                                     kda_stream_t stream) {
  using namespace kda;
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARG;
  if (B < 0 || H < 0 || T < 0 || d < 1 || x_sb < 0 || x_sh < 0 || x_st < 0)
    return KDA_ERR_INVALID_ARG;
  if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
  if ((long long)B * H == 0 || (T == 0 && !sT)) return KDA_OK;
  if (!w || (T > 0 && (!x || !y))) return KDA_ERR_INVALID_ARG;
  if (!aligned(x, size_of(dt)) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(s0, 16) ||
      !aligned(lens, 4) || !aligned(y, 16) || !aligned(sT, 16))
    return KDA_ERR_INVALID_ARG;
  const ConvArgs a{x, x_sb, x_sh, x_st, w, bias, s0, lens, y, sT, B, H, T, d, act == KDA_ACT_SILU};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dt == KDA_BF16 ? launch_conv<__nv_bfloat16>(a, W, st) : launch_conv<float>(a, W, st);
}

extern "C" kda_status kda_short_conv_step(const void *x, long long x_sn, long long x_sh,
                                          const float *w, const float *bias, void *S,
                                          const int *slots, int n_slots, void *y, int N, int H,
                                          int d, int W, kda_dtype dt, kda_act act,
                                          kda_stream_t stream) {
  using namespace kda;
  if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARG;
  if (N < 0 || H < 0 || d < 1 || n_slots < 0 || x_sn < 0 || x_sh < 0) return KDA_ERR_INVALID_ARG;
  if (!slots && N > n_slots) return KDA_ERR_INVALID_ARG;
  if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
  if ((long long)N * H == 0 || n_slots == 0) return KDA_OK;
  if (!x || !w || !S || !y) return KDA_ERR_INVALID_ARG;
  if (!aligned(x, size_of(dt)) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(S, 16) ||
      !aligned(slots, 4) || !aligned(y, 16))
    return KDA_ERR_INVALID_ARG;
  const ConvStepArgs a{x, x_sn, x_sh, w, bias, S, slots, n_slots, y, N, H, d, act == KDA_ACT_SILU};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dt == KDA_BF16 ? launch_conv_step<__nv_bfloat16>(a, W, st)
                        : launch_conv_step<float>(a, W, st);
}
