// rope.cu -- rotary positions: q and k rotated pair by pair by an angle
// proportional to their position, v copied along (the change of layout from
// a projection's token-major rows to the attention's head-major ones).
//
//   (y1, y2) = factor (x1 cos t - x2 sin t, x1 sin t + x2 cos t),
//   t = pos f_i; the backward pass is the rotation by -t.
//
// The angle.  Far positions lose a 32-bit angle (pos f at 1e6 radians keeps
// 0.06), and 64-bit arithmetic is slow here, so the frequency is kept in
// turns as a 64-bit fraction: pos * phase modulo 2^64 is an exact integer
// product whose top 32 bits are the fraction of a turn, whatever the
// position's sign; sincospi of it is right to fp32.  (The fraction's own
// rounding, 2^-65 a position, stays below fp32's to positions of 2^40.)
//
// Bound by HBM: every element is read once and written once.  A thread's
// angles serve up to 12 heads, so the sines cost 1/12 of a pair's loads, and
// two heads' loads go out before their stores.  Measured in bf16 (GB300, copy
// rate 6.77 TB/s): 131072 tokens of 28 + 4 + 4 heads of 128 354 us, 1.01 of
// the copy rate (one head's loads at a time 379 us); 4 x 8192 tokens of 32 +
// 32 + 32 heads, into a packed layout, 238 us, 1.00; interleaved pairs over
// half of the head in fp16 94 us, 0.95 (a pair to a thread, not packed 101
// us).  A call on 64 tokens takes 26 us, its host's time.
#include "layer.h"
#include "layer_vec.cuh"

namespace ra {

namespace {

constexpr int kThreads = 256;

// What the threads of a token share out: `turn` units of the rotary part, then
// the rest of a q or k head, and for v whole heads.  A unit is two packs of V
// elements; consecutive threads' first packs are adjacent, and so are their
// second ones.
struct Units {
  int turn, qk, v, all;
};

// A thread owns one unit of one token for a range of heads: cos and sin of
// its V pairs stay in its registers while the heads go by.
template <typename T, int V, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, const Units n, int heads_per_cta) {
  const long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long tok = id / n.all;
  if (tok >= static_cast<long long>(a.B) * a.L) return;
  const int u = static_cast<int>(id - tok * n.all);
  const int b = static_cast<int>(tok / a.L), l = static_cast<int>(tok - static_cast<long long>(b) * a.L);
  const bool turn = u < n.turn;
  // the unit's two packs in a q or k head, and whether they are there: the
  // pairs' first and second elements, packs of whole pairs (two elements at
  // V = 1), or two of the rest
  int e0, e1;
  bool has0 = u < n.qk, has1 = has0;
  constexpr bool kPacked = kInter && V > 1;  // pairs within a pack
  if (turn) {
    e0 = kInter && V == 1 ? 2 * u : V * u;
    e1 = !kInter ? a.R / 2 + V * u : V == 1 ? 2 * u + 1 : V * (u + n.turn);
    if (kPacked) has1 = e1 < a.R;
  } else {
    e0 = a.R + V * (u - n.turn);
    e1 = e0 + V * (n.qk - n.turn);
    has1 = has1 && e1 < a.d;
  }
  float c[V], s[V];
  if (turn) {
    long long pos;
    if (a.pos) {
      const long long at = b * a.pos_b + l;
      pos = a.pos64 ? static_cast<const int64_t*>(a.pos)[at] : static_cast<const int32_t*>(a.pos)[at];
    } else {
      pos = l < a.split ? a.base0 + a.step * l : a.base1 + a.step * (l - a.split);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      // pair j of the unit: of a pack of whole pairs V / 2 belong to each pack
      const int i = !kPacked ? V * u + j : j < V / 2 ? e0 / 2 + j : e1 / 2 + j - V / 2;
      const uint64_t turns = i < a.R / 2 ? a.phase[i] * static_cast<uint64_t>(pos) : 0;
      const float t = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;  // half turns, [-1, 1]
      sincospif(t, &s[j], &c[j]);
      c[j] *= a.factor;
      s[j] *= a.inverse ? -a.factor : a.factor;
    }
  }
  auto rotate = [&](Pack<T, V>& p, Pack<T, V>& q) {
    if constexpr (kPacked) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float x1 = to_f32(p.e[2 * j]), x2 = to_f32(p.e[2 * j + 1]);
        p.e[2 * j] = from_f32<T>(x1 * c[j] - x2 * s[j]);
        p.e[2 * j + 1] = from_f32<T>(x1 * s[j] + x2 * c[j]);
        const float y1 = to_f32(q.e[2 * j]), y2 = to_f32(q.e[2 * j + 1]);
        q.e[2 * j] = from_f32<T>(y1 * c[V / 2 + j] - y2 * s[V / 2 + j]);
        q.e[2 * j + 1] = from_f32<T>(y1 * s[V / 2 + j] + y2 * c[V / 2 + j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x1 = to_f32(p.e[j]), x2 = to_f32(q.e[j]);
        p.e[j] = from_f32<T>(x1 * c[j] - x2 * s[j]);
        q.e[j] = from_f32<T>(x1 * s[j] + x2 * c[j]);
      }
    }
  };
  const int lo = static_cast<int>(blockIdx.y) * heads_per_cta, hi = lo + heads_per_cta;
  int first = 0;
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    const RopeTensor& x = a.t[t];
    const int h0 = max(lo - first, 0), h1 = min(hi - first, x.H);
    first += x.H;
    if (h0 >= h1) continue;
    if (t == 2) {  // v: the copy's packs
      e0 = V * u;
      e1 = V * (u + n.v);
      has0 = u < n.v;
      has1 = has0 && e1 < a.d;
    }
    const bool turned = turn && t < 2;
    if (!has0 || (!turned && x.in == x.out)) continue;
    const T* p = static_cast<const T*>(x.in) + b * x.ib + l * x.il + h0 * x.ih;
    T* o = static_cast<T*>(x.out) + b * x.ob + l * x.ol + h0 * x.oh;
    int h = h0;
    // two heads' loads before their stores (which may be in place: the
    // compiler would not pass one by the other)
    for (; h + 1 < h1; h += 2, p += 2 * x.ih, o += 2 * x.oh) {
      Pack<T, V> v0 = load_pack<T, V>(p + e0), w0 = load_pack<T, V>(p + x.ih + e0), v1{}, w1{};
      if (has1) {
        v1 = load_pack<T, V>(p + e1);
        w1 = load_pack<T, V>(p + x.ih + e1);
      }
      if (turned) {
        rotate(v0, v1);
        rotate(w0, w1);
      }
      store_pack<T, V>(o + e0, v0);
      if (has1) store_pack<T, V>(o + e1, v1);
      store_pack<T, V>(o + x.oh + e0, w0);
      if (has1) store_pack<T, V>(o + x.oh + e1, w1);
    }
    if (h < h1) {
      Pack<T, V> v0 = load_pack<T, V>(p + e0), v1{};
      if (has1) v1 = load_pack<T, V>(p + e1);
      if (turned) rotate(v0, v1);
      store_pack<T, V>(o + e0, v0);
      if (has1) store_pack<T, V>(o + e1, v1);
    }
  }
}

template <typename T, int V>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  Units n;
  n.turn = a.interleaved && V > 1 ? (a.R / V + 1) / 2 : a.R / (2 * V);
  n.qk = n.turn + ((a.d - a.R) / V + 1) / 2;
  n.v = (a.d / V + 1) / 2;
  n.all = n.qk > n.v ? n.qk : n.v;
  const long long tokens = static_cast<long long>(a.B) * a.L;
  const long long bx = (tokens * n.all + kThreads - 1) / kThreads;
  const int heads = a.t[0].H + a.t[1].H + a.t[2].H;
  // four CTAs an SM before a thread takes more than one head, at most 12:
  // its angles are then shared by that many, and few tokens spread over all SMs
  long long per = heads * bx / (4LL * a.n_sms);
  per = per < 1 ? 1 : per > 12 ? 12 : per;
  if ((heads + per - 1) / per > 65535) per = (heads + 65534) / 65535;
  if (bx > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>((heads + per - 1) / per));
  if (a.interleaved)
    rope_kernel<T, V, true><<<grid, kThreads, 0, stream>>>(a, n, static_cast<int>(per));
  else
    rope_kernel<T, V, false><<<grid, kThreads, 0, stream>>>(a, n, static_cast<int>(per));
  return cudaGetLastError();
}

// The widest pack that every offset allows: both halves of the rotary part (of
// interleaved pairs the whole) and the rest of the head whole packs, every
// stride a multiple of it, every base aligned to its bytes.
int widest(const RopeArgs& a) {
  const int sz = dtype_bytes(a.dtype);
  for (int V = 16 / sz; V > 1; V /= 2) {
    bool ok = (a.interleaved ? a.R : a.R / 2) % V == 0 && (a.d - a.R) % V == 0;
    for (const RopeTensor& x : a.t) {
      if (!x.H) continue;
      ok = ok && reinterpret_cast<uintptr_t>(x.in) % (V * sz) == 0 && reinterpret_cast<uintptr_t>(x.out) % (V * sz) == 0;
      for (long long s : {x.ib, x.ih, x.il, x.ob, x.oh, x.ol}) ok = ok && s % V == 0;
    }
    if (ok) return V;
  }
  return 1;
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t stream) {
  switch (widest(a)) {
    case 8:
      if constexpr (sizeof(T) == 2) return launch<T, 8>(a, stream);
      return cudaErrorInvalidValue;
    case 4: return launch<T, 4>(a, stream);
    case 2: return launch<T, 2>(a, stream);
    default: return launch<T, 1>(a, stream);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.dtype == kBf16) return launch_t<__nv_bfloat16>(a, stream);
  if (a.dtype == kFp16) return launch_t<__half>(a, stream);
  return launch_t<float>(a, stream);
}

}  // namespace ra
