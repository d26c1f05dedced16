// capi_layer.cu -- the C ABI of the layer operators around the attention
// (include/ring_attn.h): rotary positions, the norms before and after a
// block with its gate and residual scale, the gradient norm and clipping.
// Argument checks and launches; the library keeps nothing between calls.
#include <algorithm>
#include <climits>
#include <cmath>
#include <map>
#include <mutex>
#include <vector>

#include "../../include/ring_attn.h"
#include "capi_internal.h"
#include "layer.h"

namespace ra {
namespace {

std::map<int, int> g_sm_counts;  // device -> multiprocessors

// Multiprocessors of the current device (caller holds g_mutex).
int sm_count(int* n) {
  int dev;
  int rc = current_device(&dev);
  if (rc != RING_ATTN_OK) return rc;
  auto it = g_sm_counts.find(dev);
  if (it == g_sm_counts.end()) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return RING_ATTN_ERR_CUDA;
    it = g_sm_counts.emplace(dev, v).first;
  }
  *n = it->second;
  return RING_ATTN_OK;
}

bool dtype_ok(int t) { return t >= kBf16 && t <= kFp32; }
bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr long long kMaxSpan = 1LL << 46;  // elements: every offset, in bytes too, stays within 64 bits

// Whether n elements `stride` apart stay within kMaxSpan.
bool stride_ok(long long n, long long stride) {
  return n <= 1 || (stride >= 0 && (stride == 0 || n - 1 <= kMaxSpan / stride));
}

// A 2- to 4-dimensional view in memory: base, bytes an element, extents and
// strides in elements.
struct View {
  const void* p;
  int size;
  long long n[4];
  long long s[4];
};

// Whether no two elements of the view share an address: with the strides in
// rising order, each is past the span of those below it.
bool injective(const View& v) {
  std::pair<long long, long long> d[4];  // stride, extent
  int k = 0;
  for (int i = 0; i < 4; ++i)
    if (v.n[i] > 1) d[k++] = {v.s[i], v.n[i]};
  std::sort(d, d + k);
  long long span = 1;
  for (int i = 0; i < k; ++i) {
    if (d[i].first < span) return false;
    span += d[i].first * (d[i].second - 1);
  }
  return true;
}

long long span_bytes(const View& v) {
  long long e = 1;
  for (int i = 0; i < 4; ++i) e += (v.n[i] - 1) * v.s[i];
  return e * v.size;
}

bool same(const View& a, const View& b) {
  if (a.p != b.p || a.size != b.size) return false;
  for (int i = 0; i < 4; ++i)
    if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.s[i] != b.s[i])) return false;
  return true;
}

// Whether two views may share memory.  Views whose spans meet are told apart
// where both repeat with one stride (the tokens of a packed buffer) and
// keep to different parts of it.
bool meet(const View& a, const View& b) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  if (pa + span_bytes(a) <= pb || pb + span_bytes(b) <= pa) return false;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      if (a.n[i] < 2 || b.n[j] < 2) continue;
      const long long st = a.s[i] * a.size;
      if (st != b.s[j] * b.size) continue;
      // bytes that each takes within one stride, whatever longer strides
      // (whole multiples of it) add
      long long wa = a.size, wb = b.size;
      bool whole = true;
      for (int k = 0; k < 4; ++k) {
        if (a.n[k] > 1 && a.s[k] * a.size < st) wa += (a.n[k] - 1) * a.s[k] * a.size;
        else if (a.n[k] > 1 && a.s[k] * a.size % st) whole = false;
        if (b.n[k] > 1 && b.s[k] * b.size < st) wb += (b.n[k] - 1) * b.s[k] * b.size;
        else if (b.n[k] > 1 && b.s[k] * b.size % st) whole = false;
      }
      if (!whole) continue;
      const long long off = static_cast<long long>((pb % st + st - pa % st) % st);  // b's part, after a's start
      if (off >= wa && off + wb <= st) return false;
    }
  return true;
}

View rows_view(const void* p, int dt, long long M, int D, long long ld) {
  return {p, dtype_bytes(dt), {1, 1, M, D}, {0, 0, M > 1 ? ld : D, 1}};
}

// Every written view apart from every other written one and from every read
// one, but for the pairs that may be the same memory.
struct Reads { View v; int same_as; };  // index of the written view it may be, or -1

int check_views(const View* w, int nw, const Reads* r, int nr) {
  for (int i = 0; i < nw; ++i) {
    if (!w[i].p) continue;
    if (!injective(w[i])) return RING_ATTN_ERR_UNSUPPORTED;
    for (int j = i + 1; j < nw; ++j)
      if (w[j].p && meet(w[i], w[j])) return RING_ATTN_ERR_UNSUPPORTED;
    for (int j = 0; j < nr; ++j) {
      if (!r[j].v.p) continue;
      if (r[j].same_as == i && same(w[i], r[j].v)) continue;
      if (meet(w[i], r[j].v)) return RING_ATTN_ERR_UNSUPPORTED;
    }
  }
  return RING_ATTN_OK;
}

struct Timed {  // brackets a call's launches while profiling is on
  LaunchTimer* t;
  int kind;
  cudaStream_t stream;
  Timed(int k, cudaStream_t s) : t(active_timer()), kind(k), stream(s) {
    if (t) t->mark(kind, false, stream);
  }
  ~Timed() {
    if (t) t->mark(kind, true, stream);
  }
};

int rope(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* v_out, const long long* strides,
         int B, int Hq, int Hkv, int L, int d, int rotary_dim, int dtype, int interleaved, int inverse,
         const uint64_t* phase, float factor, const void* positions, int positions_bytes, long long positions_batch,
         const long long* position_map, cudaStream_t stream) {
  if (B < 0 || Hq < 0 || Hkv < 0 || L < 0 || d <= 0 || rotary_dim < 0 || rotary_dim > d || rotary_dim % 2)
    return RING_ATTN_ERR_SHAPE;
  if (!dtype_ok(dtype) || d > 1024 || L > (1 << 29)) return RING_ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * L > (1LL << 40) / d || Hq > 65535 || Hkv > 65535) return RING_ATTN_ERR_UNSUPPORTED;
  if (positions && positions_bytes != 4 && positions_bytes != 8) return RING_ATTN_ERR_UNSUPPORTED;
  if (positions && !stride_ok(B, positions_batch)) return RING_ATTN_ERR_SHAPE;
  if (!positions && position_map && (position_map[0] < 0 || position_map[0] > L)) return RING_ATTN_ERR_SHAPE;
  if (!std::isfinite(factor)) return RING_ATTN_ERR_SHAPE;
  if (B == 0 || L == 0) return RING_ATTN_OK;
  if (!strides || (!phase && rotary_dim > 0)) return RING_ATTN_ERR_NULL;
  if ((!q != !q_out) || (!k != !k_out) || (!v != !v_out) || (!q && !k && !v)) return RING_ATTN_ERR_NULL;
  const int size = dtype_bytes(dtype);
  RopeArgs a;
  const void* in[3] = {q, k, v};
  void* out[3] = {q_out, k_out, v_out};
  View w[3];
  Reads r[5];
  r[3] = {View{positions, positions_bytes, {1, 1, B, L}, {0, 0, B > 1 ? positions_batch : 0, 1}}, -1};
  r[4] = {View{phase, 8, {1, 1, 1, rotary_dim / 2}, {0, 0, 0, 1}}, -1};
  for (int i = 0; i < 3; ++i) {
    RopeTensor& t = a.t[i];
    const int H = i == 0 ? Hq : Hkv;
    const long long* si = strides + 3 * i;       // batch, head, token
    const long long* so = strides + 9 + 3 * i;
    w[i] = r[i].v = View{nullptr, size, {1, 1, 1, 1}, {0, 0, 0, 0}};
    r[i].same_as = i;
    if (!in[i] || H == 0) continue;
    const long long n[] = {B, H, L};
    for (int j = 0; j < 3; ++j)
      if (!stride_ok(n[j], si[j]) || !stride_ok(n[j], so[j])) return RING_ATTN_ERR_UNSUPPORTED;
    if (!aligned_to(in[i], size) || !aligned_to(out[i], size)) return RING_ATTN_ERR_UNSUPPORTED;
    t.in = in[i];
    t.out = out[i];
    t.H = H;
    // the stride of an extent of one says nothing
    t.ib = B > 1 ? si[0] : 0; t.ih = H > 1 ? si[1] : 0; t.il = L > 1 ? si[2] : 0;
    t.ob = B > 1 ? so[0] : 0; t.oh = H > 1 ? so[1] : 0; t.ol = L > 1 ? so[2] : 0;
    r[i].v = View{in[i], size, {B, H, L, d}, {t.ib, t.ih, t.il, 1}};
    w[i] = View{out[i], size, {B, H, L, d}, {t.ob, t.oh, t.ol, 1}};
  }
  if (!a.t[0].H && !a.t[1].H && !a.t[2].H) return RING_ATTN_OK;
  int rc = check_views(w, 3, r, rotary_dim > 0 ? 5 : 4);
  if (rc != RING_ATTN_OK) return rc;
  // in place is element by element the same memory, not only the same base
  for (int i = 0; i < 3; ++i)
    if (a.t[i].H && a.t[i].in == a.t[i].out && !same(w[i], r[i].v)) return RING_ATTN_ERR_UNSUPPORTED;
  if (!aligned_to(phase, 8) || (positions && !aligned_to(positions, positions_bytes))) return RING_ATTN_ERR_UNSUPPORTED;
  a.B = B; a.L = L; a.d = d; a.R = rotary_dim;
  a.dtype = dtype; a.interleaved = interleaved != 0; a.inverse = inverse;
  a.phase = phase; a.factor = factor;
  a.pos = positions; a.pos64 = positions_bytes == 8; a.pos_b = positions_batch;
  a.split = L;
  if (!positions && position_map) {
    a.split = static_cast<int>(position_map[0]);
    a.base0 = position_map[1];
    a.base1 = position_map[2];
    a.step = position_map[3];
  }
  std::lock_guard<std::mutex> lock(g_mutex);
  if ((rc = sm_count(&a.n_sms)) != RING_ATTN_OK) return rc;
  Timed t(RING_ATTN_KERNEL_ROPE, stream);
  return launch_rope(a, stream) == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ERR_CUDA;
}

int check_norm(long long M, int D, long long gate_rows, int dt_x, int dt_a, int dt_gate, int flags, float scale) {
  if (M < 0 || D <= 0 || gate_rows < 0 || (flags & ~15)) return RING_ATTN_ERR_SHAPE;
  if (gate_rows > 0 && M > 0 && (gate_rows > M || M % gate_rows)) return RING_ATTN_ERR_SHAPE;
  if (!std::isfinite(scale)) return RING_ATTN_ERR_SHAPE;
  if (D > kNormMaxD || M > (1LL << 40)) return RING_ATTN_ERR_UNSUPPORTED;
  if (!dtype_ok(dt_x) || !dtype_ok(dt_a) || (dt_x != dt_a && dt_x != kFp32)) return RING_ATTN_ERR_UNSUPPORTED;
  if (gate_rows > 0 && dt_gate != kFp32 && dt_gate != dt_a) return RING_ATTN_ERR_UNSUPPORTED;
  return RING_ATTN_OK;
}

bool ld_ok(const void* p, long long ld, int D, long long M) {
  return !p || M <= 1 || (ld >= D && stride_ok(M, ld));
}

View vec_view(const void* p, int D) { return rows_view(p, kFp32, 1, D, D); }

// Addresses that a call writes (out) or reads, for the overlap check.
struct Range {
  uintptr_t lo, hi;
  bool out;
};

int check_grads(const void* const* grads, void* const* outs, const long long* n, const int* dt, const int* dt_out,
                int n_tensors, const Range* own, int n_own, std::vector<GradTensor>* list) {
  if (n_tensors == 0) return RING_ATTN_OK;
  if (!grads || !n || !dt) return RING_ATTN_ERR_NULL;
  list->resize(n_tensors);
  long long total = 0;  // (a launch counts its chunks in 32 bits)
  for (int i = 0; i < n_tensors; ++i) {
    if (n[i] < 0) return RING_ATTN_ERR_SHAPE;
    if (!dtype_ok(dt[i]) || (dt_out && !dtype_ok(dt_out[i])) || n[i] > (1LL << 40)) return RING_ATTN_ERR_UNSUPPORTED;
    if ((total += n[i]) > (1LL << 44)) return RING_ATTN_ERR_UNSUPPORTED;
    GradTensor& g = (*list)[i];
    g = {grads[i], outs ? outs[i] : nullptr, n[i], dt[i], dt_out ? dt_out[i] : dt[i]};
    if (n[i] == 0) continue;
    if (!g.in || (outs && !g.out)) return RING_ATTN_ERR_NULL;
    if (!aligned_to(g.in, dtype_bytes(g.dt_in)) || (outs && !aligned_to(g.out, dtype_bytes(g.dt_out))))
      return RING_ATTN_ERR_UNSUPPORTED;
  }
  // Each output, the norm and the workspace apart from one another and from
  // every gradient but an output's own, which it may be (same memory, same
  // type).
  std::vector<Range> w;
  w.reserve(2 * static_cast<size_t>(n_tensors) + n_own);
  for (int i = 0; i < n_tensors; ++i) {
    const GradTensor& g = (*list)[i];
    if (g.n == 0) continue;
    const uintptr_t in = reinterpret_cast<uintptr_t>(g.in), out = reinterpret_cast<uintptr_t>(g.out);
    if (outs) w.push_back({out, out + g.n * dtype_bytes(g.dt_out), true});
    if (outs && g.in == g.out && g.dt_in == g.dt_out) continue;
    w.push_back({in, in + g.n * dtype_bytes(g.dt_in), false});
  }
  // (views of one buffer come in order: then a pass over them is enough)
  auto below = [](const Range& a, const Range& b) { return a.lo < b.lo; };
  if (!std::is_sorted(w.begin(), w.end(), below)) std::sort(w.begin(), w.end(), below);
  for (int i = 0; i < n_own; ++i) w.insert(std::upper_bound(w.begin(), w.end(), own[i], below), own[i]);
  // in rising order: the ends reached so far by outputs and by gradients
  uintptr_t out_end = 0, in_end = 0;
  for (const Range& r : w) {
    if (r.lo < out_end || (r.out && r.lo < in_end)) return RING_ATTN_ERR_UNSUPPORTED;
    uintptr_t& end = r.out ? out_end : in_end;
    end = std::max(end, r.hi);
  }
  return RING_ATTN_OK;
}

enum class Clip { kNorm, kScale, kBoth };

int grads_run(Clip what, const void* const* grads, void* const* outs, const long long* n, const int* dt,
              const int* dt_out, int n_tensors, float max_norm, float* norm, void* ws, size_t ws_bytes,
              cudaStream_t stream) {
  std::vector<GradTensor> list;
  if (what != Clip::kNorm && !(max_norm >= 0.f)) return RING_ATTN_ERR_SHAPE;
  if (what != Clip::kNorm && n_tensors > 0 && !outs) return RING_ATTN_ERR_NULL;
  if (n_tensors < 0) return RING_ATTN_ERR_SHAPE;
  if (!norm) return RING_ATTN_ERR_NULL;
  if (!aligned_to(norm, 4)) return RING_ATTN_ERR_UNSUPPORTED;
  const size_t need = what == Clip::kScale ? 0 : grad_workspace_bytes(n_tensors);
  if (need && (!ws || ws_bytes < need || !aligned_to(ws, 256))) return RING_ATTN_ERR_WORKSPACE;
  const uintptr_t pn = reinterpret_cast<uintptr_t>(norm), pw = reinterpret_cast<uintptr_t>(ws);
  const Range own[2] = {{pn, pn + 4, true}, {pw, pw + need, true}};
  int rc = check_grads(grads, outs, n, dt, dt_out, n_tensors, own, need ? 2 : 1, &list);
  if (rc != RING_ATTN_OK) return rc;
  GradArgs a;
  a.tensors = list.data();
  a.n_tensors = n_tensors;
  a.max_norm = max_norm;
  a.norm = norm;
  a.partial = static_cast<double*>(ws);
  std::lock_guard<std::mutex> lock(g_mutex);
  Timed t(RING_ATTN_KERNEL_GRAD_CLIP, stream);
  const cudaError_t e = what == Clip::kNorm    ? launch_grad_norm(a, stream)
                        : what == Clip::kScale ? launch_grad_scale(a, stream)
                                               : launch_grad_clip(a, stream);
  return e == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ERR_CUDA;
}

// No C++ exception leaves a C entry.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return RING_ATTN_ERR_CUDA;
  }
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" {

int ring_attn_rope_fwd(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* v_out,
                       const long long* strides, int B, int Hq, int Hkv, int L, int d, int rotary_dim, int dtype,
                       int interleaved, const uint64_t* phase, float factor, const void* positions,
                       int positions_bytes, long long positions_batch, const long long* position_map,
                       cudaStream_t stream) {
  return guarded([&] {
    return rope(q, k, v, q_out, k_out, v_out, strides, B, Hq, Hkv, L, d, rotary_dim, dtype, interleaved, 0, phase,
                factor, positions, positions_bytes, positions_batch, position_map, stream);
  });
}

int ring_attn_rope_bwd(const void* dq, const void* dk, const void* dv, void* dq_out, void* dk_out, void* dv_out,
                       const long long* strides, int B, int Hq, int Hkv, int L, int d, int rotary_dim, int dtype,
                       int interleaved, const uint64_t* phase, float factor, const void* positions,
                       int positions_bytes, long long positions_batch, const long long* position_map,
                       cudaStream_t stream) {
  return guarded([&] {
    return rope(dq, dk, dv, dq_out, dk_out, dv_out, strides, B, Hq, Hkv, L, d, rotary_dim, dtype, interleaved, 1, phase,
                factor, positions, positions_bytes, positions_batch, position_map, stream);
  });
}

int ring_attn_block_norm_fwd(const void* x, const void* a, const float* post_w, const float* post_b, const void* gate,
                             const float* pre_w, const float* pre_b, void* y, void* h, float* stats,
                             const long long* row_strides, long long M, int D, long long gate_rows, int dtype_x,
                             int dtype_a, int dtype_gate, int flags, float scale, float eps, cudaStream_t stream) {
  return guarded([&] {
    int rc = check_norm(M, D, gate_rows, dtype_x, dtype_a, dtype_gate, flags, scale);
    if (rc != RING_ATTN_OK) return rc;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return static_cast<int>(RING_ATTN_ERR_SHAPE);
    if (M == 0) return static_cast<int>(RING_ATTN_OK);
    const bool post = flags & kNormPost, pre = flags & kNormPre;
    // nothing to compute, or a post norm, gate or y without a block's output
    if (!a && (post || gate || gate_rows || y || !pre)) return static_cast<int>(RING_ATTN_ERR_SHAPE);
    // weights of a norm that is not taken, a bias of a root-mean-square norm
    if ((!post && (post_w || post_b)) || (!pre && (pre_w || pre_b || h)) || (!(flags & kNormLayer) && (post_b || pre_b)))
      return static_cast<int>(RING_ATTN_ERR_SHAPE);
    if (!x || !row_strides || !stats || (a && !y) || (pre && !h) || (gate_rows > 0) != (gate != nullptr))
      return static_cast<int>(RING_ATTN_ERR_NULL);
    const long long* ld = row_strides;  // x, a, gate, y, h
    const void* ptr[] = {x, a, gate, y, h};
    const int dt[] = {dtype_x, dtype_a, dtype_gate, dtype_x, dtype_a};
    for (int i = 0; i < 5; ++i) {
      if (!ld_ok(ptr[i], ld[i], D, i == 2 ? gate_rows : M)) return static_cast<int>(RING_ATTN_ERR_SHAPE);
      if (!aligned_to(ptr[i], dtype_bytes(ptr[i] ? dt[i] : kBf16))) return static_cast<int>(RING_ATTN_ERR_UNSUPPORTED);
    }
    for (const float* p : {post_w, post_b, pre_w, pre_b, static_cast<const float*>(stats)})
      if (!aligned_to(p, 4)) return static_cast<int>(RING_ATTN_ERR_UNSUPPORTED);
    const int ns = (flags & kNormLayer) ? 4 : 2;
    const View w[] = {rows_view(y, dtype_x, M, D, ld[3]), rows_view(h, dtype_a, M, D, ld[4]),
                      View{stats, 4, {1, 1, ns, M}, {0, 0, M, 1}}};
    const Reads r[] = {{rows_view(x, dtype_x, M, D, ld[0]), 0},
                       {rows_view(a, dtype_a, M, D, ld[1]), 1},
                       {rows_view(gate, dtype_gate, gate_rows ? gate_rows : 1, D, ld[2]), -1},
                       {vec_view(post_w, D), -1},
                       {vec_view(post_b, D), -1},
                       {vec_view(pre_w, D), -1},
                       {vec_view(pre_b, D), -1}};
    if ((rc = check_views(w, 3, r, 7)) != RING_ATTN_OK) return rc;
    BlockNormArgs p;
    p.x = x; p.a = a; p.gate = gate;
    p.post_w = post_w; p.post_b = post_b; p.pre_w = pre_w; p.pre_b = pre_b;
    p.y = y; p.h = h; p.stats = stats;
    p.ld_x = ld[0]; p.ld_a = ld[1]; p.ld_gate = ld[2]; p.ld_y = ld[3]; p.ld_h = ld[4];
    if (M == 1) p.ld_x = p.ld_a = p.ld_y = p.ld_h = 0;
    if (gate_rows <= 1) p.ld_gate = 0;
    p.M = M; p.D = D; p.gate_rows = gate_rows; p.flags = flags;
    p.dt_x = dtype_x; p.dt_a = dtype_a; p.dt_gate = dtype_gate;
    p.scale = scale; p.eps = eps;
    std::lock_guard<std::mutex> lock(g_mutex);
    if ((rc = sm_count(&p.n_sms)) != RING_ATTN_OK) return rc;
    Timed t(RING_ATTN_KERNEL_BLOCK_NORM, stream);
    return static_cast<int>(launch_block_norm_fwd(p, stream) == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ERR_CUDA);
  });
}

size_t ring_attn_block_norm_bwd_workspace_size(long long M, int D, long long gate_rows, int flags) {
  if (check_norm(M, D, gate_rows, kFp32, kFp32, kFp32, flags, 1.f) != RING_ATTN_OK) return 0;
  return M == 0 ? 0 : block_norm_bwd_workspace(M, D, gate_rows, flags);
}

int ring_attn_block_norm_bwd(const void* dy, const void* dh, const void* y, const void* a, const float* stats,
                             const float* post_w, const float* post_b, const void* gate, const float* pre_w, void* dx,
                             void* da, void* dgate, float* dpost_w, float* dpost_b, float* dpre_w, float* dpre_b,
                             const long long* row_strides, long long M, int D, long long gate_rows, int dtype_x,
                             int dtype_a, int dtype_gate, int flags, float scale, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
  return guarded([&] {
    int rc = check_norm(M, D, gate_rows, dtype_x, dtype_a, dtype_gate, flags, scale);
    if (rc != RING_ATTN_OK) return rc;
    float* sums[] = {dpost_w, dpost_b, dpre_w, dpre_b};
    if (M == 0) {  // sums over no rows, the shared gate's fp32 ones among them
      if (gate_rows > (1LL << 40)) return static_cast<int>(RING_ATTN_ERR_UNSUPPORTED);
      auto clear = [&](void* s, long long rows) {
        return !s || rows == 0 || cudaMemsetAsync(s, 0, static_cast<size_t>(rows) * D * 4, stream) == cudaSuccess;
      };
      for (void* s : {static_cast<void*>(dpost_w), static_cast<void*>(dpost_b), static_cast<void*>(dpre_w),
                      static_cast<void*>(dpre_b), dgate})
        if (!aligned_to(s, 4)) return static_cast<int>(RING_ATTN_ERR_UNSUPPORTED);
      for (float* s : sums)
        if (!clear(s, 1)) return static_cast<int>(RING_ATTN_ERR_CUDA);
      return static_cast<int>(clear(dgate, gate_rows) ? RING_ATTN_OK : RING_ATTN_ERR_CUDA);
    }
    const bool post = flags & kNormPost, pre = flags & kNormPre, layer = flags & kNormLayer;
    const bool shared = gate_rows > 0 && gate_rows < M;
    if (!a && (post || gate || gate_rows || da || dgate || !pre)) return static_cast<int>(RING_ATTN_ERR_SHAPE);
    if (!post && (post_w || post_b || dpost_w || dpost_b)) return static_cast<int>(RING_ATTN_ERR_SHAPE);
    if (!pre && (pre_w || dpre_w || dpre_b || dh || y)) return static_cast<int>(RING_ATTN_ERR_SHAPE);
    if (!layer && (post_b || dpost_b || dpre_b)) return static_cast<int>(RING_ATTN_ERR_SHAPE);
    // a gradient for each weight, a gate and its gradient
    if ((post_w && !dpost_w) || (pre_w && !dpre_w) || (gate_rows > 0) != (dgate != nullptr))
      return static_cast<int>(RING_ATTN_ERR_NULL);
    if (!row_strides || !stats || !dx || (pre && (!dh || !y)) || (!pre && !dy) || (a && !da) ||
        (gate_rows > 0) != (gate != nullptr))
      return static_cast<int>(RING_ATTN_ERR_NULL);
    const long long* ld = row_strides;  // dy, dh, y, a, gate, dx, da
    const void* ptr[] = {dy, dh, y, a, gate, dx, da};
    const int dt[] = {dtype_x, dtype_a, dtype_x, dtype_a, dtype_gate, dtype_x, dtype_a};
    for (int i = 0; i < 7; ++i) {
      if (!ld_ok(ptr[i], ld[i], D, i == 4 ? gate_rows : M)) return static_cast<int>(RING_ATTN_ERR_SHAPE);
      if (!aligned_to(ptr[i], dtype_bytes(ptr[i] ? dt[i] : kBf16))) return static_cast<int>(RING_ATTN_ERR_UNSUPPORTED);
    }
    const int dt_dgate = shared ? static_cast<int>(kFp32) : dtype_gate;
    for (const float* p : {post_w, post_b, pre_w, stats, static_cast<const float*>(dpost_w),
                           static_cast<const float*>(dpost_b), static_cast<const float*>(dpre_w),
                           static_cast<const float*>(dpre_b)})
      if (!aligned_to(p, 4)) return static_cast<int>(RING_ATTN_ERR_UNSUPPORTED);
    if (dgate && !aligned_to(dgate, dtype_bytes(dt_dgate))) return static_cast<int>(RING_ATTN_ERR_UNSUPPORTED);
    const size_t need = block_norm_bwd_workspace(M, D, gate_rows, flags);
    if (!workspace || workspace_bytes < need || !aligned_to(workspace, 256))
      return static_cast<int>(RING_ATTN_ERR_WORKSPACE);
    const int ns = layer ? 4 : 2;
    const View w[] = {rows_view(dx, dtype_x, M, D, ld[5]),
                      rows_view(da, dtype_a, M, D, ld[6]),
                      rows_view(dgate, dt_dgate, gate_rows ? gate_rows : 1, D, D),
                      vec_view(dpost_w, D),
                      vec_view(dpost_b, D),
                      vec_view(dpre_w, D),
                      vec_view(dpre_b, D),
                      View{workspace, 1, {1, 1, 1, static_cast<long long>(need)}, {0, 0, 0, 1}}};
    const Reads r[] = {{rows_view(dy, dtype_x, M, D, ld[0]), 0},
                       {rows_view(dh, dtype_a, M, D, ld[1]), 1},
                       {rows_view(y, dtype_x, M, D, ld[2]), -1},
                       {rows_view(a, dtype_a, M, D, ld[3]), -1},
                       {rows_view(gate, dtype_gate, gate_rows ? gate_rows : 1, D, ld[4]), -1},
                       {View{stats, 4, {1, 1, ns, M}, {0, 0, M, 1}}, -1},
                       {vec_view(post_w, D), -1},
                       {vec_view(post_b, D), -1},
                       {vec_view(pre_w, D), -1}};
    if ((rc = check_views(w, 8, r, 9)) != RING_ATTN_OK) return rc;
    BlockNormArgs p;
    p.dy = dy; p.dh = dh; p.y = const_cast<void*>(y); p.a = a; p.gate = gate;
    p.stats = const_cast<float*>(stats);
    p.post_w = post_w; p.post_b = post_b; p.pre_w = pre_w;
    p.dx = dx; p.da = da; p.dgate = dgate;
    p.dpost_w = dpost_w; p.dpost_b = dpost_b; p.dpre_w = dpre_w; p.dpre_b = dpre_b;
    p.ld_dy = ld[0]; p.ld_dh = ld[1]; p.ld_y = ld[2]; p.ld_a = ld[3]; p.ld_gate = ld[4]; p.ld_dx = ld[5]; p.ld_da = ld[6];
    if (M == 1) p.ld_dy = p.ld_dh = p.ld_y = p.ld_a = p.ld_dx = p.ld_da = 0;
    if (gate_rows <= 1) p.ld_gate = 0;
    p.M = M; p.D = D; p.gate_rows = gate_rows; p.flags = flags;
    p.dt_x = dtype_x; p.dt_a = dtype_a; p.dt_gate = dtype_gate;
    p.scale = scale;
    p.partial = static_cast<float*>(workspace);
    std::lock_guard<std::mutex> lock(g_mutex);
    Timed t(RING_ATTN_KERNEL_BLOCK_NORM, stream);
    return static_cast<int>(launch_block_norm_bwd(p, stream) == cudaSuccess ? RING_ATTN_OK : RING_ATTN_ERR_CUDA);
  });
}

size_t ring_attn_grad_workspace_size(int n_tensors) { return n_tensors < 0 ? 0 : grad_workspace_bytes(n_tensors); }

int ring_attn_grad_norm(const void* const* grads, const long long* n_elems, const int* dtypes, int n_tensors,
                        float* norm, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return guarded([&] {
    return grads_run(Clip::kNorm, grads, nullptr, n_elems, dtypes, nullptr, n_tensors, 0.f, norm, workspace,
                     workspace_bytes, stream);
  });
}

int ring_attn_grad_scale(const void* const* grads, void* const* outs, const long long* n_elems, const int* dtypes,
                         const int* out_dtypes, int n_tensors, float max_norm, const float* norm, cudaStream_t stream) {
  return guarded([&] {
    return grads_run(Clip::kScale, grads, outs, n_elems, dtypes, out_dtypes, n_tensors, max_norm,
                     const_cast<float*>(norm), nullptr, 0, stream);
  });
}

int ring_attn_grad_clip(const void* const* grads, void* const* outs, const long long* n_elems, const int* dtypes,
                        const int* out_dtypes, int n_tensors, float max_norm, float* norm, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  return guarded([&] {
    return grads_run(Clip::kBoth, grads, outs, n_elems, dtypes, out_dtypes, n_tensors, max_norm, norm, workspace,
                     workspace_bytes, stream);
  });
}

}  // extern "C"
