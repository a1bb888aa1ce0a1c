// kda_state.cu -- copies and clears of whole states between the slots of a
// pool: compaction, forks and fresh slots of a cache of fixed-size states.
//
// The lists come from the host and travel in the launch's arguments, so a
// call needs no device copy of them, checks every index before it launches
// and can be captured.  Pairs none of which touches what another writes run at
// once; the effect of the list's order is kept by starting a new launch, which
// the stream orders, where a pair does.  A list that would take many launches
// (a shift of all slots by one) runs in one, in which each thread takes its
// bytes of a slot through all pairs in order.
//
// HBM bounds a copy of large states: 48 states of 2 MiB in 32.9 us, 6.1 TB/s of
// the 201 MB read and written (0.92 of a copy).
#include <stdint.h>

#include "kda_launch.cuh"

namespace kda {
namespace {

constexpr int kStateThreads = 256;
constexpr int kPieces = 4;      // loads in flight per thread
constexpr int kMaxPairs = 448;  // pairs per launch: 3.5 KiB of launch arguments
// Launches of a batch of pairs; more go in order in one (a shift of 64 slots of 2 MiB by one:
// 55 us, where the bytes take 40; of 256 slots of 24 KiB: 50 us).
constexpr int kMaxLaunches = 4;

struct PairList {
  int src[kMaxPairs], dst[kMaxPairs];
};

// V: the widest type that divides the pool's address, strides and slots.
template <typename V>
__global__ void __launch_bounds__(kStateThreads)
state_copy_kernel(const __grid_constant__ PairList list, char *pool, long long layer_stride,
                  long long slot_bytes) {
  char *layer = pool + blockIdx.z * layer_stride;
  const V *s = reinterpret_cast<const V *>(layer + list.src[blockIdx.y] * slot_bytes);
  V *d = reinterpret_cast<V *>(layer + list.dst[blockIdx.y] * slot_bytes);
  const long long n = slot_bytes / (long long)sizeof(V);
  const long long i0 = (long long)blockIdx.x * (kStateThreads * kPieces) + threadIdx.x;
  V v[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
    if (i0 + k * kStateThreads < n) v[k] = s[i0 + k * kStateThreads];
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
    if (i0 + k * kStateThreads < n) d[i0 + k * kStateThreads] = v[k];
}

// Pairs 0 to n - 1 one after the other: every thread moves the same bytes of each
// slot, so its own order is the order of the list.
template <typename V>
__global__ void __launch_bounds__(kStateThreads)
state_copy_ordered_kernel(const __grid_constant__ PairList list, int n, char *pool,
                          long long layer_stride, long long slot_bytes) {
  char *layer = pool + blockIdx.z * layer_stride;
  const long long i = (long long)blockIdx.x * kStateThreads + threadIdx.x;
  if (i >= slot_bytes / (long long)sizeof(V)) return;
  for (int k = 0; k < n; ++k) {
    const V v = reinterpret_cast<const V *>(layer + list.src[k] * slot_bytes)[i];
    reinterpret_cast<V *>(layer + list.dst[k] * slot_bytes)[i] = v;
  }
}

template <typename V>
__global__ void __launch_bounds__(kStateThreads)
state_clear_kernel(const __grid_constant__ PairList list, char *pool, long long layer_stride,
                   long long slot_bytes) {
  V *d = reinterpret_cast<V *>(pool + blockIdx.z * layer_stride +
                               list.dst[blockIdx.y] * slot_bytes);
  const long long n = slot_bytes / (long long)sizeof(V);
  const long long i0 = (long long)blockIdx.x * (kStateThreads * kPieces) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
    if (i0 + k * kStateThreads < n) d[i0 + k * kStateThreads] = V{};
}

enum Kind { kCopy, kCopyOrdered, kClear };

template <typename V>
kda_status launch_batch(const PairList &list, int n, Kind kind, char *pool, int layers,
                        long long layer_stride, long long slot_bytes, cudaStream_t st) {
  const long long per = (long long)kStateThreads * (kind == kCopyOrdered ? 1 : kPieces) * sizeof(V);
  const long long chunks = (slot_bytes + per - 1) / per;
  if (chunks > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  for (int l = 0; l < layers; l += 65535) {
    const dim3 grid((unsigned)chunks, kind == kCopyOrdered ? 1 : n,
                    layers - l < 65535 ? layers - l : 65535);
    char *p = pool + l * layer_stride;
    if (kind == kCopy)
      state_copy_kernel<V><<<grid, kStateThreads, 0, st>>>(list, p, layer_stride, slot_bytes);
    else if (kind == kCopyOrdered)
      state_copy_ordered_kernel<V>
          <<<grid, kStateThreads, 0, st>>>(list, n, p, layer_stride, slot_bytes);
    else
      state_clear_kernel<V><<<grid, kStateThreads, 0, st>>>(list, p, layer_stride, slot_bytes);
  }
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status run_batch(const PairList &list, int n, Kind kind, char *pool, int layers,
                     long long layer_stride, long long slot_bytes, cudaStream_t st) {
  if (n == 0) return KDA_OK;
  const uintptr_t a = reinterpret_cast<uintptr_t>(pool) | (uintptr_t)layer_stride |
                      (uintptr_t)slot_bytes;
  if (a % 16 == 0)
    return launch_batch<uint4>(list, n, kind, pool, layers, layer_stride, slot_bytes, st);
  if (a % 4 == 0)
    return launch_batch<uint32_t>(list, n, kind, pool, layers, layer_stride, slot_bytes, st);
  if (a % 2 == 0)
    return launch_batch<uint16_t>(list, n, kind, pool, layers, layer_stride, slot_bytes, st);
  return launch_batch<uint8_t>(list, n, kind, pool, layers, layer_stride, slot_bytes, st);
}

// Slots that the current batch reads and writes: an open-addressing table on
// the stack, at most 2 kMaxPairs of its entries in use.
struct Touched {
  static constexpr int kSize = 2048;
  int key[kSize];  // slot + 1, 0: free
  unsigned char use[kSize];  // 1 read, 2 written
  Touched() { clear(); }
  void clear() {
    for (int i = 0; i < kSize; ++i) key[i] = 0;
  }
  unsigned char &at(int slot) {
    unsigned i = ((unsigned)slot * 2654435761u) >> 21;
    while (key[i] != 0 && key[i] != slot + 1) i = (i + 1) % kSize;
    if (key[i] == 0) {
      key[i] = slot + 1;
      use[i] = 0;
    }
    return use[i];
  }
};

kda_status check_pool(const void *pool, int layers, long long layer_stride, int n_slots,
                      long long slot_bytes, const int *a, const int *b, int n) {
  if (layers < 0 || n_slots < 0 || slot_bytes < 0 || n < 0 || layer_stride < 0)
    return KDA_ERR_INVALID_ARG;
  if (n_slots > 0 && slot_bytes > (1LL << 62) / n_slots) return KDA_ERR_INVALID_ARG;
  if (layers > 1 && layer_stride < n_slots * slot_bytes) return KDA_ERR_INVALID_ARG;
  if (n > 0 && (!a || !b)) return KDA_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (a[i] < 0 || a[i] >= n_slots || b[i] < 0 || b[i] >= n_slots) return KDA_ERR_INVALID_ARG;
  if (n > 0 && layers > 0 && slot_bytes > 0 && !pool) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

}  // namespace
}  // namespace kda

extern "C" kda_status kda_state_copy(void *pool, int layers, long long layer_stride, int n_slots,
                                     long long slot_bytes, const int *src, const int *dst, int n,
                                     kda_stream_t stream) {
  using namespace kda;
  const kda_status ok = check_pool(pool, layers, layer_stride, n_slots, slot_bytes, src, dst, n);
  if (ok != KDA_OK) return ok;
  if (layers == 0 || slot_bytes == 0) return KDA_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (layers == 1) layer_stride = 0;
  char *p = static_cast<char *>(pool);
  Touched touched;
  for (int i = 0; i < n;) {
    // up to kMaxPairs pairs that do something, and where a new launch has to begin
    PairList list;
    int start[kMaxLaunches + 1], launches = 1, m = 0;
    start[0] = 0;
    touched.clear();
    for (; i < n && m < kMaxPairs; ++i) {
      if (src[i] == dst[i]) continue;
      if (launches <= kMaxLaunches && ((touched.at(src[i]) & 2) || touched.at(dst[i]) != 0)) {
        if (launches < kMaxLaunches) start[launches] = m;
        ++launches;
        touched.clear();
      }
      if (launches <= kMaxLaunches) {
        touched.at(src[i]) |= 1;
        touched.at(dst[i]) |= 2;
      }
      list.src[m] = src[i];
      list.dst[m++] = dst[i];
    }
    if (launches > kMaxLaunches) {
      const kda_status e =
          run_batch(list, m, kCopyOrdered, p, layers, layer_stride, slot_bytes, st);
      if (e != KDA_OK) return e;
      continue;
    }
    start[launches] = m;
    for (int l = 0; l < launches; ++l) {
      PairList part;
      const int k = start[l + 1] - start[l];
      for (int j = 0; j < k; ++j)
        part.src[j] = list.src[start[l] + j], part.dst[j] = list.dst[start[l] + j];
      const kda_status e = run_batch(part, k, kCopy, p, layers, layer_stride, slot_bytes, st);
      if (e != KDA_OK) return e;
    }
  }
  return KDA_OK;
}

extern "C" kda_status kda_state_clear(void *pool, int layers, long long layer_stride, int n_slots,
                                      long long slot_bytes, const int *slots, int n,
                                      kda_stream_t stream) {
  using namespace kda;
  const kda_status ok =
      check_pool(pool, layers, layer_stride, n_slots, slot_bytes, slots, slots, n);
  if (ok != KDA_OK) return ok;
  if (layers == 0 || slot_bytes == 0) return KDA_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (layers == 1) layer_stride = 0;
  PairList list;
  for (int i = 0; i < n; i += kMaxPairs) {
    const int m = n - i < kMaxPairs ? n - i : kMaxPairs;
    for (int k = 0; k < m; ++k) list.src[k] = list.dst[k] = slots[i + k];
    const kda_status e = run_batch(list, m, kClear, static_cast<char *>(pool), layers,
                                   layer_stride, slot_bytes, st);
    if (e != KDA_OK) return e;
  }
  return KDA_OK;
}
