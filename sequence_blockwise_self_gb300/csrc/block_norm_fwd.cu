// block_norm_fwd.cu -- the forward of the block norms (block_norm.cuh).
#include "block_norm.cuh"

namespace ra {
namespace norm {
namespace {

// 16 columns a thread.  Measured at 131072 x 3584 in bf16: eight columns and
// one group of 14 warps a CTA 731 us, that with two rows a step (one barrier
// for both) 673 us, one row a step in two such CTAs an SM 615 us, 16 columns
// in two groups 558 us: 0.99 of the copy rate.  (Over inputs that change from
// call to call 574 us, 0.97.)
constexpr int V = 2;
constexpr int kMost = 768, kGroups = 12;  // threads and groups of several warps of a CTA
constexpr size_t kAhead = 60 * 1024;      // bytes fetched ahead

// Where a row's gate comes from: folded into the weights (none, or one gate
// row), the ring (one per token, or for a few rows), the thread's own shared
// memory (one for many rows), or memory row by row where those have no room.
enum GateFrom : int { kFolded, kRing, kKept, kDirect };

// The weights are in shared memory once a CTA, for all its groups: w of the
// pre norm, A, for layer norms their b and B, 32 slots to a plane, a warp's
// planes together (a thread's next plane is at a constant distance, and
// groups of part of a warp read the same slots).  A stage of the ring: a row
// of x, a and, at kRing, the gate.
template <typename Tx, typename Ta, bool kVec, bool kLayer, bool kNarrow>
__global__ void __launch_bounds__(kMost)
    block_norm_fwd_kernel(const BlockNormArgs p, int threads, int groups, int stages, int gate_from) {
  extern __shared__ uint4 smem[];
  const int D = p.D, group = static_cast<int>(threadIdx.x) / threads;
  const int tid = static_cast<int>(threadIdx.x) - group * threads, lane = tid & 31;  // of the group's
  const float inv_d = 1.f / static_cast<float>(D);
  const bool post = p.flags & kNormPost, pre = p.flags & kNormPre, sig = p.flags & kNormGateSigmoid;
  const bool has_a = p.a != nullptr;
  const long long per_gate = p.gate ? p.M / p.gate_rows : p.M;  // rows of one gate row
  int col[V];
#pragma unroll
  for (int i = 0; i < V; ++i) col[i] = kVec ? 8 * (tid + i * threads) : 8 * (V * tid + i);
  // (barrier 0 is the CTA's)
  const uint32_t mask = group_mask<kNarrow>(threads);
  constexpr int kBuf = kLayer ? RowMoments<kNarrow>::kBuf : 32;
  __shared__ __align__(16) float bufs[kGroups * kBuf];
  __shared__ float counts[16];
  RowSum<1, kNarrow> sum{bufs + kBuf * (group % kGroups), mask, threads, tid >> 5, group + 1, 0};
  RowMoments<kNarrow> moments{bufs + kBuf * (group % kGroups), mask, threads, tid >> 5, group + 1, 0, 0.f, 0.f, 0, 0.f};
  for (int k = threadIdx.x; k < kGroups * kBuf; k += blockDim.x) bufs[k] = 0.f;

  constexpr int kWeights = kLayer ? 16 : 8;  // planes: four to a weight
  uint4* const w_pre = smem + (tid >> 5) * 32 * kWeights + lane;
  uint4* const w_post = w_pre + 4 * 32;
  uint4* const b_pre = w_pre + 8 * 32;   // layer norms
  uint4* const b_post = w_pre + 12 * 32;
  constexpr int plane = 32;
  const int kept_planes = gate_from == kKept ? 4 : 0, my_warp = static_cast<int>(threadIdx.x) >> 5;
  uint4* const kept = smem + (threads + 31) / 32 * 32 * kWeights + my_warp * 32 * kept_planes + (threadIdx.x & 31);  // a gate row's columns
  constexpr int kA = kRowPlanes<Tx, V, kVec>, kG = kA + kRowPlanes<Ta, V, kVec>;
  const int stage_step = (kG + (gate_from == kRing ? (p.dt_gate == kFp32 ? kRowPlanes<float, V, kVec> : kRowPlanes<Ta, V, kVec>) : 0)) * plane;
  uint4* const ring = kept + ((static_cast<int>(blockDim.x) + 31) / 32 - my_warp) * 32 * kept_planes + my_warp * stages * stage_step;
  if (col[V - 1] + 8 > D)  // columns past D are never fetched, and read as zero
    for (int k = 0; k < stages * stage_step; k += plane) ring[k] = make_uint4(0, 0, 0, 0);

  // the rows of a group are every `workers`th: at any time the CTAs are on
  // neighbouring rows
  const long long worker = static_cast<long long>(blockIdx.x) * groups + group, workers = static_cast<long long>(gridDim.x) * groups;
  // (from the ring with rows that share one: 32 bits hold them)
  auto gate_row = [&](long long r) {
    return per_gate == 1 ? r : static_cast<long long>(static_cast<uint32_t>(r) / static_cast<uint32_t>(per_gate));
  };
  auto fetch = [&](long long r, uint4* at) {
    if (r < p.M) {
      fetch_cols<Tx, kVec>(at, plane, static_cast<const Tx*>(p.x), static_cast<const Tx*>(p.x) + r * p.ld_x, col, D);
      if (has_a) fetch_cols<Ta, kVec>(at + kA * plane, plane, static_cast<const Ta*>(p.a), static_cast<const Ta*>(p.a) + r * p.ld_a, col, D);
      if (gate_from == kRing) {
        const long long g = gate_row(r);
        if (p.dt_gate == kFp32) fetch_cols<float, kVec>(at + kG * plane, plane, static_cast<const float*>(p.gate), static_cast<const float*>(p.gate) + g * p.ld_gate, col, D);
        else fetch_cols<Ta, kVec>(at + kG * plane, plane, static_cast<const Ta*>(p.gate), static_cast<const Ta*>(p.gate) + g * p.ld_gate, col, D);
      }
    }
    cp_commit();
  };
  for (int s = 0; s < stages - 1; ++s) fetch(worker + s * workers, ring + s * stage_step);
  if (kLayer) moments.begin(col, D, counts);
  // y = x + norm(a) A + B with A = scale w, B = scale b, times g where there
  // is one gate row (others multiply them row by row)
  if (group == 0) {
    Cols f[V], w[V];
    if (p.gate && gate_from == kFolded) gate_cols<Ta, kVec>(p, 0, col, f);
    else for (int i = 0; i < V; ++i) f[i] = all_cols(1.f);
    auto put = [&](uint4* to, const float* weight, float absent, bool scaled) {
      weight_cols<kVec>(weight, col, D, absent, w);
      if (scaled)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) w[i].p[j] = mul2(w[i].p[j], mul2(f[i].p[j], both(p.scale)));
      put_cols(to, 32, w);
    };
    put(w_pre, p.pre_w, 1.f, false);
    put(w_post, p.post_w, 1.f, true);
    if (kLayer) {
      put(b_pre, p.pre_b, 0.f, false);
      put(b_post, p.post_b, 0.f, true);
    }
  }
  __syncthreads();
  if (kLayer) moments.finish(counts);
  long long gate_end = 0;  // first row past the gate row that is kept
  // v -> its norm before the weights; (mean, rstd)
  auto normed = [&](Cols (&v)[V]) {
    float2 st;
    float off = 0.f;
    if constexpr (kLayer) {
      const float3 m = moments.template operator()<V, kVec>(v, col, D);
      st = make_float2(m.x, rsqrtf(m.y * inv_d + p.eps));
      off = m.z * st.y;
    } else {
      float2 t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t[i] = both(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) t[i] = fma2(v[i].p[j], v[i].p[j], t[i]);
        if (i > 0) t[0] = add2(t[0], t[i]);
      }
      float s[1] = {sum2(t[0])};
      sum(s);
      st = make_float2(0.f, rsqrtf(s[0] * inv_d + p.eps));
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].p[j] = kLayer ? fma2(v[i].p[j], both(st.y), both(off)) : mul2(v[i].p[j], both(st.y));
    return st;
  };
  // v -> v w [+ b], of weights in shared memory
  auto weighted = [&](Cols (&v)[V], const uint4* at_w, const uint4* at_b) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Cols w = weight_at(at_w, 32, i), b = kLayer ? weight_at(at_b, 32, i) : all_cols(0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].p[j] = kLayer ? fma2(v[i].p[j], w.p[j], b.p[j]) : mul2(v[i].p[j], w.p[j]);
    }
  };

  int stage = 0;
  for (long long r = worker; r < p.M; r += workers) {
    const uint4* at = ring + stage * stage_step;
    fetch(r + (stages - 1) * workers, ring + (stage == 0 ? stages - 1 : stage - 1) * stage_step);
    cp_wait(stages - 1);
    Cols x[V];
    take_cols<Tx, kVec>(at, plane, x, shift_of<Tx, kVec>(static_cast<const Tx*>(p.x) + r * p.ld_x));
    float2 st1 = both(0.f), st2 = both(0.f);
    if (has_a) {
      Cols a[V];
      take_cols<Ta, kVec>(at + kA * plane, plane, a, shift_of<Ta, kVec>(static_cast<const Ta*>(p.a) + r * p.ld_a));
      if (post) st1 = normed(a);
      weighted(a, w_post, b_post);
      if (gate_from != kFolded) {
        Cols w[V];
        if (gate_from == kRing) {
          const long long g = kVec ? 0 : gate_row(r);
          if (p.dt_gate == kFp32)
            take_cols<float, kVec>(at + kG * plane, plane, w, shift_of<float, kVec>(static_cast<const float*>(p.gate) + g * p.ld_gate));
          else
            take_cols<Ta, kVec>(at + kG * plane, plane, w, shift_of<Ta, kVec>(static_cast<const Ta*>(p.gate) + g * p.ld_gate));
#pragma unroll
          for (int i = 0; i < V; ++i) gate_value(w[i], sig);
        } else if (gate_from == kKept && r < gate_end) {
          take_cols<float, true>(kept, plane, w, 0);
        } else {
          gate_cols<Ta, kVec>(p, r / per_gate, col, w);
          if (gate_from == kKept) {
            put_cols(kept, plane, w);
            gate_end = (r / per_gate + 1) * per_gate;
          }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) a[i].p[j] = mul2(a[i].p[j], w[i].p[j]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i].p[j] = add2(x[i].p[j], a[i].p[j]);
      store_cols<Tx, kVec>(static_cast<Tx*>(p.y) + r * p.ld_y, col, D, x, mask);
    }
    if (pre) {
      // h takes y before its rounding to the stream's type: one rounding
      st2 = normed(x);
      weighted(x, w_pre, b_pre);
      store_cols<Ta, kVec>(static_cast<Ta*>(p.h) + r * p.ld_h, col, D, x, mask);
    }
    if (tid == 0) {
      p.stats[r] = st1.y;
      p.stats[p.M + r] = st2.y;
      if (kLayer) {
        p.stats[2 * p.M + r] = st1.x;
        p.stats[3 * p.M + r] = st2.x;
      }
    }
    stage = stage + 1 < stages ? stage + 1 : 0;
  }
}

}  // namespace
}  // namespace norm

cudaError_t launch_block_norm_fwd(const BlockNormArgs& a, cudaStream_t stream) {
  using namespace norm;
  const bool vec = a.D % 8 == 0 && vec_ok(a.x, a.ld_x, a.dt_x) && vec_ok(a.a, a.ld_a, a.dt_a) &&
                   vec_ok(a.gate, a.ld_gate, a.dt_gate) && vec_ok(a.y, a.ld_y, a.dt_x) && vec_ok(a.h, a.ld_h, a.dt_a) &&
                   vec_ok(a.post_w, 0, kFp32) && vec_ok(a.post_b, 0, kFp32) && vec_ok(a.pre_w, 0, kFp32) &&
                   vec_ok(a.pre_b, 0, kFp32);
  const bool layer_norm = a.flags & kNormLayer;
  const int threads = threads_for(a.D, V);
  auto row_planes = [&](int dt) { return V * dtype_bytes(dt) / 2 + (vec ? 0 : 1); };  // kRowPlanes
  const size_t weights = static_cast<size_t>(threads + 31) / 32 * 32 * 16 * (layer_norm ? 16 : 8);
  GateFrom gate_from = kFolded;
  // A gate row that a group keeps is waited for when it changes, one from the
  // ring is not, but is asked for by all groups that share it at once: kept
  // from one and a half rows of a group on (32768 x 3584, 456 groups, layer
  // norm: 256 rows of a gate row kept 268 us, from the ring 202 us, 1024 rows
  // 219 and 203 us; 9993 x 1000, 1672 groups, 3331 rows: 32 and 42 us).  The
  // rows of a group alone do not part the two sides: 1024 rows, 2.2 of a group,
  // are kept although the ring would be faster, for the sake of 3331 rows, 2.0
  // of a group, where it is slower.
  if (a.gate && a.gate_rows > 1) {
    const long long rows = a.M / a.gate_rows, most = static_cast<long long>(a.n_sms) * (kMost / threads);
    gate_from = rows == 1 || (2 * rows < 3 * most && a.M <= 0xffffffffLL) ? kRing : kKept;
  }
  // Groups of a CTA.  Where a row takes long -- a layer norm's two sums,
  // rows of part accesses, a gate row beside it, a group too small to hide its
  // own waits -- as many as the registers allow (32768 x 3584, groups x
  // stages: layer norm 3 x 2 178 us against 2 x 2 215 us; rows of 3583 247
  // against 275 us; gates of 4096 rows 143 against 163 us).  Else up to 512
  // threads, or two groups (32768 x 5120: one 254 us, two 200 us): with
  // more, reads and writes crowd each other out (2 x 3 140 us, 3 x 2 153 us,
  // 3 x 3 164 us).
  const bool slow = layer_norm || !vec || gate_from == kKept || threads <= 64;
  int groups = slow ? kMost / threads : std::max(512 / threads, std::min(2, kMost / threads));
  // no more of them than shorten the longest run of rows
  const long long runs = (a.M + a.n_sms - 1) / a.n_sms;
  const long long steps = (runs + groups - 1) / groups;
  groups = static_cast<int>((runs + steps - 1) / steps);
  size_t fixed, stage;
  auto sizes = [&] {
    const size_t plane = static_cast<size_t>(threads * groups + 31) / 32 * 32 * 16;
    fixed = weights + (gate_from == kKept ? 4 * plane : 0);
    stage = (row_planes(a.dt_x) + row_planes(a.dt_a) + (gate_from == kRing ? row_planes(a.dt_gate) : 0)) * plane;
  };
  // as many of them as leave room for two stages, and without a layer norm's
  // pauses no more than 70 KB in one (300000 x 200 in fp32 147 us with 64 KB,
  // 185 us with 96 KB)
  for (sizes(); groups > 1 && (fixed + 2 * stage > kSmem || (!layer_norm && groups > 2 && stage > 70 * 1024)); sizes()) --groups;
  if (fixed + stage > kSmem) {
    gate_from = kDirect;
    sizes();
  }
  const unsigned ctas = static_cast<unsigned>(std::min<long long>((a.M + groups - 1) / groups, a.n_sms));
  // Stages: 60 KB ahead of the rows at hand, or one row; a lone group two
  // rows.  More crowd the writes out: 32768 x 3584 in fp32 292 us with one
  // row ahead (57 KB), 375 us with two; 65536 x 2048 in bf16, four groups,
  // 162 us with one (33 KB), 183 us with two.
  const size_t ahead = std::max<size_t>(kAhead / stage, groups == 1 ? 2 : 1);
  const int stages = stages_for(stage, std::min(kSmem - fixed, (ahead + 1) * stage));
  if (fixed + stages * stage > kSmem) return cudaErrorInvalidValue;
  auto run = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<ctas, threads * groups, fixed + stages * stage, stream>>>(a, threads, groups, stages, gate_from);
    return cudaGetLastError();
  };
  return by_types(a, [&](auto x, auto y) {
    using Tx = decltype(x);
    using Ta = decltype(y);
    auto narrow = [&](auto whole, auto layer) {
      return threads < 32 ? run(block_norm_fwd_kernel<Tx, Ta, whole(), layer(), true>)
                          : run(block_norm_fwd_kernel<Tx, Ta, whole(), layer(), false>);
    };
    const std::true_type yes;
    const std::false_type no;
    if (layer_norm) return vec ? narrow(yes, yes) : narrow(no, yes);
    return vec ? narrow(yes, no) : narrow(no, no);
  });
}

}  // namespace ra
