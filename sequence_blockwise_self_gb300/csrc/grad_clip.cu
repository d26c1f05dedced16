// grad_clip.cu -- the global norm of many gradient tensors and their
// clipping: n = sqrt(sum over all tensors of g^2), out = g min(1, max / n).
//
// Two launches over the same chunks of the tensors' elements: the first
// leaves one fp64 sum of squares per CTA, the second adds them (every CTA
// in the same order, so all use the same norm and two runs give the same
// bits) and scales.  A gradient is read twice -- the norm has to be known
// before the first write -- the second time back to front, where L2 still
// holds what the first launch read last.
//
// Bound by HBM.  Measured: 103 M fp32 elements to bf16 158 us, 822 MB read and
// 206 MB written less what L2 keeps (of the first reading's 411 MB about 42
// MB): 0.92 of the copy rate (183 us before four loads in flight and the back
// to front order); 401 bf16 tensors of 100 M elements at odd offsets 102 us on
// the GPU (109 us with eight CTAs an SM and every chunk's ends element by
// element), as long as the host takes for their addresses.  Chunks of 4096
// elements instead of 16384: 198 us.  Streaming hints on the second launch's
// loads and stores: no gain.  A small clipping takes 6 to 9 us in a graph, two
// launches; the second starts while the first ends.
#include <algorithm>
#include <type_traits>

#include "layer.h"
#include "layer_vec.cuh"

namespace ra {

namespace {

constexpr int kThreads = 256;
constexpr long long kChunk = 16384;  // elements
constexpr int kMaxCtas = 608;  // partial sums of one launch: four an SM of a GB300, on any device (the sums' order)
constexpr long long kKeptBytes = 80LL << 20;  // of the L2, between the launches

// The tensors of one launch, in the kernel's parameters: no copy to the
// device, and a captured graph keeps them.
template <int N>
struct Table {
  const void* in[N];
  void* out[N];
  long long n[N];
  int first[N + 1];  // chunk of the tensor's first element
  uint8_t dt[N];     // input type | output type << 2
  int count;
};
constexpr int kSmall = 32, kMiddle = 256, kLarge = 1024;
static_assert(sizeof(Table<kLarge>) < 32000, "kernel parameters");

// The tensor of chunk c: the last one whose first chunk is not past it.
template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int c) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double cta_sum(double v, double* buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.;
  for (int w = 0; w < kThreads / 32; ++w) s += buf[w];
  return s;
}

// Elements of [p, p + n) in front of the first aligned 16 bytes.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  const int h = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / static_cast<int>(sizeof(T));
  return h < n ? h : n;
}

// 16 bytes; kLast: this launch is their last reader (evicted first).
template <typename T, bool kLast>
__device__ __forceinline__ Pack<T, 16 / sizeof(T)> load16(const T* p) {
  Pack<T, 16 / sizeof(T)> r;
  const uint4 w = kLast ? __ldcs(reinterpret_cast<const uint4*>(p)) : *reinterpret_cast<const uint4*>(p);
  *reinterpret_cast<uint4*>(&r) = w;
  return r;
}

// Sum of (mul g)^2 over this thread's elements of [g, g + n): aligned packs,
// and element by element what is in front of them and behind.
template <typename T, bool kLast>
__device__ float squares(const T* g, int n, float mul) {
  constexpr int E = 16 / sizeof(T);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  const int head = head_of(g, n), packs = (n - head) / E, tail = head + packs * E;
#pragma unroll 8
  for (int k = threadIdx.x; k < packs; k += kThreads) {
    const auto p = load16<T, kLast>(g + head + k * E);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float x = to_f32(p.e[j]) * mul;
      s[j & 3] += x * x;
    }
  }
  const int rest = head + (n - tail);  // below 16
  if (static_cast<int>(threadIdx.x) < rest) {
    const int k = static_cast<int>(threadIdx.x) < head ? threadIdx.x : tail + (threadIdx.x - head);
    const float x = to_f32(g[k]) * mul;
    s[0] += x * x;
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// The same as fp64, in range for every finite value: a sum that overflowed,
// or is so small that squares may have been lost, is taken again scaled by a
// power of two.
template <typename T>
__device__ double safe_squares(const T* g, int n, bool last) {
  const float s = last ? squares<T, true>(g, n, 1.f) : squares<T, false>(g, n, 1.f);
  if (!(s <= 0x1p120f)) return static_cast<double>(squares<T, false>(g, n, 0x1p-70f)) * 0x1p140;
  if (s < 0x1p-60f) return static_cast<double>(squares<T, false>(g, n, 0x1p90f)) * 0x1p-180;
  return s;
}

// Elements [lo, hi) of chunk c of a tensor of n elements, the first of them
// c kChunk: but for the tensor's own ends at its first 16-byte boundaries.
struct Span {
  long long lo;
  int n;
};
template <typename T>
__device__ __forceinline__ Span span_of(const T* p, int c, long long n) {
  const long long at = c * kChunk;
  const int shift = head_of(p, 16);
  const long long lo = c ? at + shift : 0, hi = min(at + kChunk + shift, n);
  return {lo, static_cast<int>(max(hi - lo, 0LL))};
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) grad_squares_kernel(const __grid_constant__ Table<N> t, double* partial, int keep_from) {
  __shared__ double buf[kThreads / 32];
  double sum = 0.;
  for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const bool last = c < keep_from;  // gone from L2 before the second launch comes to it
    auto add = [&](auto p) {
      const Span at = span_of(p, c - t.first[k], t.n[k]);
      sum += safe_squares(p + at.lo, at.n, last);
    };
    switch (t.dt[k] & 3) {
      case kBf16: add(static_cast<const __nv_bfloat16*>(t.in[k])); break;
      case kFp16: add(static_cast<const __half*>(t.in[k])); break;
      default: add(static_cast<const float*>(t.in[k])); break;
    }
  }
  sum = cta_sum(sum, buf);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// out = g c d with d = 1, or where max / n is below 2^-100 c = 2^100 max / n
// and d = 2^-100: a subnormal factor would have lost bits that the product
// has.  (There max is below 2^28 and n above 2^-49, but for a max of 0:
// nothing on the way leaves the range, and c is at most 1.)
struct Factor {
  float c, d;
  __device__ __forceinline__ float operator()(float g) const { return g * c * d; }
};
__device__ __forceinline__ Factor factor_of(float max_norm, float n) {
  const float c = max_norm / n;
  if (c >= 0x1p-100f || max_norm == 0.f) return {c, 1.f};
  return {max_norm * 0x1p64f / (n * 0x1p-36f), 0x1p-100f};
}

// o = f(g): packs of V elements, 16 bytes of the wider type (a warp's accesses
// to both are consecutive), from its first aligned one on, where the other
// type's is aligned too; else by element.
template <typename T, typename U>
__device__ void scale_chunk(const T* g, U* o, int n, Factor f) {
  constexpr int V = 16 / (sizeof(T) > sizeof(U) ? sizeof(T) : sizeof(U));
  int head = sizeof(T) > sizeof(U) ? head_of(g, n) : head_of(o, n);
  if (reinterpret_cast<uintptr_t>(g + head) % (V * sizeof(T)) || reinterpret_cast<uintptr_t>(o + head) % (V * sizeof(U))) head = n;
  const int packs = (n - head) / V, tail = head + packs * V;
  using In = std::conditional_t<V * sizeof(T) == 16, uint4, uint2>;
  using Out = std::conditional_t<V * sizeof(U) == 16, uint4, uint2>;
  const In* from = reinterpret_cast<const In*>(g + head);
  Out* to = reinterpret_cast<Out*>(o + head);
  auto scaled = [&](In w) {
    Pack<T, V> p;
    Pack<U, V> q;
    *reinterpret_cast<In*>(&p) = w;
#pragma unroll
    for (int j = 0; j < V; ++j) q.e[j] = from_f32<U>(f(to_f32(p.e[j])));
    return *reinterpret_cast<Out*>(&q);
  };
  // four loads before their stores (which might be to the same memory: the
  // compiler would not pass one by the other)
  int k = threadIdx.x;
  for (; k + 3 * kThreads < packs; k += 4 * kThreads) {
    const In a = from[k], b = from[k + kThreads], d = from[k + 2 * kThreads], e = from[k + 3 * kThreads];
    to[k] = scaled(a);
    to[k + kThreads] = scaled(b);
    to[k + 2 * kThreads] = scaled(d);
    to[k + 3 * kThreads] = scaled(e);
  }
  for (; k < packs; k += kThreads) to[k] = scaled(from[k]);
  for (k = threadIdx.x; k < head + (n - tail); k += kThreads) {
    const int at = k < head ? k : tail + (k - head);
    o[at] = from_f32<U>(f(to_f32(g[at])));
  }
}

template <typename T>
__device__ void scale_to(const T* g, void* out, int dt, int chunk, long long n, Factor f) {
  auto scale = [&](auto o) {
    const Span at = sizeof(*g) > sizeof(*o) ? span_of(g, chunk, n) : span_of(o, chunk, n);
    scale_chunk(g + at.lo, o + at.lo, at.n, f);
  };
  switch (dt) {
    case kBf16: scale(static_cast<__nv_bfloat16*>(out)); break;
    case kFp16: scale(static_cast<__half*>(out)); break;
    default: scale(static_cast<float*>(out)); break;
  }
}

// partials > 0: the norm is their root sum, written to *norm by one CTA;
// else it is read from *norm.
template <int N>
__global__ void __launch_bounds__(kThreads, 4) grad_scale_kernel(const __grid_constant__ Table<N> t, const double* partial,
                                                              int partials, float* norm, float max_norm, int write_norm) {
  __shared__ double buf[kThreads / 32];
  float n;
  after_previous();
  if (partials > 0) {
    double s = 0.;
    for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
    n = static_cast<float>(sqrt(cta_sum(s, buf)));
    if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  } else {
    n = *norm;
  }
  // a norm that is not finite leaves the values as they are
  const bool clip = n > max_norm && n <= 3.402823466e38f;
  const Factor f = clip ? factor_of(max_norm, n) : Factor{1.f, 1.f};
  const int chunks = t.first[t.count];
  for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
    const int j = chunks - 1 - i;
    const int k = tensor_of(t, j);
    if (!clip && t.in[k] == t.out[k]) continue;
    const int dt = t.dt[k] >> 2, chunk = j - t.first[k];
    switch (t.dt[k] & 3) {
      case kBf16: scale_to(static_cast<const __nv_bfloat16*>(t.in[k]), t.out[k], dt, chunk, t.n[k], f); break;
      case kFp16: scale_to(static_cast<const __half*>(t.in[k]), t.out[k], dt, chunk, t.n[k], f); break;
      default: scale_to(static_cast<const float*>(t.in[k]), t.out[k], dt, chunk, t.n[k], f); break;
    }
  }
}

// The norm alone, from the partial sums.
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* partial, int partials, float* norm) {
  __shared__ double buf[kThreads / 32];
  after_previous();
  double s = 0.;
  for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
  s = cta_sum(s, buf);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <int N>
int fill(Table<N>& t, const GradArgs& a, int from) {
  int k = 0;
  long long chunks = 0;
  for (; k < N && from + k < a.n_tensors; ++k) {
    const GradTensor& g = a.tensors[from + k];
    t.in[k] = g.in;
    t.out[k] = g.out;
    t.n[k] = g.n;
    t.dt[k] = static_cast<uint8_t>(g.dt_in | g.dt_out << 2);
    t.first[k] = static_cast<int>(chunks);
    chunks += (g.n + kChunk - 1) / kChunk;
  }
  t.first[k] = static_cast<int>(chunks);
  t.count = k;
  return k;
}

int ctas_for(int chunks) { return chunks < 1 ? 1 : chunks < kMaxCtas ? chunks : kMaxCtas; }

// The launches over all tensors, at most N to each.
template <int N>
cudaError_t squares_all(const GradArgs& a, bool keep, int* partials, cudaStream_t stream) {
  Table<N> t;
  *partials = 0;
  for (int from = 0; from < a.n_tensors;) {
    from += fill(t, a, from);
    const int ctas = ctas_for(t.first[t.count]);
    // what the second launch reads first, back to front, is kept in L2: the
    // last chunks of the last table
    long long kept = 0;
    int keep_from = t.first[t.count];
    if (from == a.n_tensors)
      for (int k = t.count; k-- > 0 && kept < kKeptBytes;) {
        const long long size = dtype_bytes(t.dt[k] & 3), chunks = t.first[k + 1] - t.first[k];
        const long long take = std::min(chunks, (kKeptBytes - kept) / (kChunk * size) + 1);
        keep_from = t.first[k + 1] - static_cast<int>(take);
        kept += take * kChunk * size;
      }
    grad_squares_kernel<N><<<ctas, kThreads, 0, stream>>>(t, a.partial + *partials, keep ? keep_from : t.first[t.count]);
    *partials += ctas;
  }
  return cudaGetLastError();
}

template <int N>
cudaError_t scale_all(const GradArgs& a, int partials, cudaStream_t stream) {
  Table<N> t;
  for (int from = (a.n_tensors - 1) / N * N; from >= 0; from -= N) {  // the last table first
    fill(t, a, from);
    const cudaError_t e = launch_after(grad_scale_kernel<N>, dim3(ctas_for(t.first[t.count])), kThreads, stream, t,
                                       a.partial, partials, a.norm, a.max_norm, from == 0 ? 1 : 0);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_workspace_bytes(int n_tensors) {
  const size_t launches = (static_cast<size_t>(n_tensors) + kLarge - 1) / kLarge;
  return (launches ? launches : 1) * kMaxCtas * sizeof(double);
}

namespace {

// f(capacity of a launch's table)
template <typename F>
cudaError_t by_count(int n, F f) {
  if (n <= kSmall) return f(std::integral_constant<int, kSmall>{});
  if (n <= kMiddle) return f(std::integral_constant<int, kMiddle>{});
  return f(std::integral_constant<int, kLarge>{});
}

}  // namespace

cudaError_t launch_grad_norm(const GradArgs& a, cudaStream_t stream) {
  int partials = 0;
  const cudaError_t e = by_count(a.n_tensors, [&](auto n) { return squares_all<n()>(a, false, &partials, stream); });
  if (e != cudaSuccess) return e;
  return launch_after(grad_norm_kernel, dim3(1), kThreads, stream, a.partial, partials, a.norm);
}

cudaError_t launch_grad_scale(const GradArgs& a, cudaStream_t stream) {
  return by_count(a.n_tensors, [&](auto n) { return scale_all<n()>(a, 0, stream); });
}

cudaError_t launch_grad_clip(const GradArgs& a, cudaStream_t stream) {
  if (a.n_tensors == 0) return launch_grad_norm(a, stream);
  int partials = 0;
  const cudaError_t e = by_count(a.n_tensors, [&](auto n) { return squares_all<n()>(a, true, &partials, stream); });
  if (e != cudaSuccess) return e;
  return by_count(a.n_tensors, [&](auto n) { return scale_all<n()>(a, partials, stream); });
}

}  // namespace ra
