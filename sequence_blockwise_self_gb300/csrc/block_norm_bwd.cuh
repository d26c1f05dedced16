// block_norm_bwd.cuh -- the backward of the block norms (block_norm.cuh).
// With t^ the normed rows before w and b and d the incoming gradients:
//
//   N:  v = d w,  dt = rstd (v - mean(v t^) t^ [- mean(v)]),
//       dw = sum d t^,  db = sum d
//   dx = dy + N_pre'(dh),  dz = scale g dx,  dg = sum scale dx z [g'],
//   da = N_post'(dz)
//
// Where rows share a gate row, sum dx a^ and sum dx over them are all that
// the weights' and the gate's gradients need: scale g and scale (w, b) are
// applied to the sums.  The sums over rows are made in one order: a thread
// adds its columns over its group's rows, a CTA its groups', the kernel
// after this one the CTAs'.
//
// Bound by HBM where the row sums let it: 32768 x 3584 in bf16 218 us, 0.96
// of the copy rate; layer
// norms, with twice the sums, 283 us (0.74), with a gate per token 20000 x
// 4096 219 us (0.88 with the gate's bytes); rows of 3583, whose accesses are
// shifted and whose sums spill, 481 us (0.43) and 662 us (layer norms).
#pragma once
#include "block_norm.cuh"

namespace ra {
namespace norm {

constexpr int kLayerThreads = 384;  // where a layer norm's sums over rows fit the registers at 16 columns
// One CTA an SM of a GB300, one row of partial sums each: fixed, so that the
// workspace and the order of the sums, and with it the bits, are the same on
// any device.  (One with fewer SMs takes the CTAs in turns.)
constexpr int kCtas = 152;

// Columns and rows at a time.  16 columns a thread and one row a step keep
// two groups of warps an SM apart at 3584 columns (32768 rows of a
// root-mean-square norm: 228 us, against 255 us with eight columns and two
// rows a step, one barrier for both).  A layer norm's four sums over rows do
// not fit 128 registers that way, and what spills falls out of the L1 that
// the ring leaves (32768 x 3584 382 us against 283 us, 20000 x 4096 with a
// gate per token 354 us against 219 us); wider than 4096 columns 16 it is,
// with 168 registers up to 6144.  And up to 256 columns half of each warp
// would idle (65536 x 256: 52 us against 37 us).
inline int packs_for(int D, bool vec, bool layer) {
  if (!vec || D > 8 * kThreads) return 2;  // (rows of part accesses: one variant)
  return layer || D <= 256 ? 1 : 2;
}

// How the rows are split among the groups.  A unit is a set of rows that
// share their gate row; units are [G][S], S to each gate row, which take its
// rows in turn, R at a time (at any time the CTAs are on neighbouring rows);
// a group takes a run of units.
struct Split {
  long long G, rows;  // gate rows that several rows share (1 if none do), rows of each
  long long S, units;
  int threads, groups, ctas;  // of a group, of a CTA, and CTAs
  bool shared;
};

// groups: at most so many to a CTA.
inline Split split_rows(long long M, int D, int V, long long gate_rows, int groups = kThreads) {
  Split s;
  s.threads = threads_for(D, V);
  // (groups of part of a warp have more statistics to keep beside their ring)
  s.groups = (s.threads < 32 ? kThreads - 64 : kThreads) / s.threads;
  s.shared = gate_rows > 0 && gate_rows < M;
  s.G = s.shared ? gate_rows : 1;
  s.rows = M / s.G;
  if (s.groups > groups) s.groups = groups;
  // groups together in a CTA once every SM has one
  const long long want = (M + kCtas - 1) / kCtas;
  if (s.groups > want) s.groups = static_cast<int>(want);
  if (s.G > 1 && s.groups > 16) s.groups = 16;  // (each leaves a row of partial sums)
  const long long most = static_cast<long long>(kCtas) * s.groups;
  s.S = most / s.G;
  const long long steps = (s.rows + 2 - V) / (3 - V);  // of R = 3 - V rows
  if (s.S > steps) s.S = steps;
  if (s.S < 1) s.S = 1;
  s.units = s.G * s.S;
  const long long used = s.units < most ? s.units : most;
  s.ctas = static_cast<int>((used + s.groups - 1) / s.groups);
  return s;
}

// Planes of a thread's columns of a row (kRowPlanes).
inline int row_planes(int dt, int V, bool vec) { return V * dtype_bytes(dt) / 2 + (vec ? 0 : 1); }

// Groups of a CTA: as many as the threads allow, but more bytes than this in
// a stage of the ring crowd HBM's reads and writes out -- sooner with a
// root-mean-square norm, whose groups come back for more sooner (groups x
// stages, stage: 65536 x 1024 in bf16 6 x 2, 49 KB, 124 us, 8 x 2, 66 KB,
// 138 us; 32768 x 2048 3 x 2, 49 KB, 127 us, 4 x 2, 66 KB, 133 us; with an
// fp32 stream 2 x 2, 49 KB, 201 us, 3 x 2, 74 KB, 184 us, 4 x 2, 98 KB, 235
// us; layer norm, 40000 x 1024, fp32 stream, 2 x 2, 49 KB, 166 us, 3 x 2, 74
// KB, 118 us, 4 x 2, 98 KB, 141 us).  Rows of part accesses are slower than
// that (30000 x 1023: 6 x 2 116 us, 8 x 1 114 us), and groups of part of a
// warp have small stages.
inline int groups_for(const BlockNormArgs& a, int V, bool vec) {
  const int threads = threads_for(a.D, V), all = kThreads / threads;
  if (!vec || threads < 32) return all;
  const bool layer = a.flags & kNormLayer, token = a.gate && a.gate_rows == a.M;
  const int planes = 2 * (row_planes(a.dt_x, V, vec) + row_planes(a.dt_a, V, vec)) + (token ? row_planes(a.dt_gate, V, vec) : 0);
  const int kb = threads * (3 - V) * planes / 64;
  int groups = (layer ? 90 : 62) / kb;
  if (groups < 3 && 3 * kb <= 75) groups = 3;
  return std::min(std::max(groups, 2), all);
}

// A row of partial sums: sum dh yhat, sum dx ahat, for layer norms sum dh and
// sum dx too, each [D].  A CTA leaves one; with several gate rows each of its
// groups does, and where a gate row's rows are split among groups, a row [D]
// of the gate's sums follows for each unit.
enum Sums : int { kPreW, kPostW, kPreB, kPostB };

struct Partials {
  int n, rows;  // sums in a row, and rows
  float* row;
  float* unit;  // [units][D]
};

// t -> t^ = (t - mean) rstd: the difference first, exact where t is near the
// mean.  (As one fma, t rstd + (-mean rstd) with that product rounded, a row
// of mean 3e4 deviations is off by up to 1e-3 in t^, for the 1 to 2 % of
// time that the difference takes: 32768 x 3584 279 against 283 us.)
template <bool kLayer>
__device__ __forceinline__ void normed(Cols& t, float mean, float rstd) {
#pragma unroll
  for (int j = 0; j < 4; ++j) t.p[j] = mul2(kLayer ? add2(t.p[j], both(-mean)) : t.p[j], both(rstd));
}

// A row's statistics, read from shared memory at this place.
__device__ __forceinline__ float4 stats_at(const float4* at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at)))
               : "memory");
  return v;
}

// Weights in shared memory, the same for every row of a unit, each thread's
// own: w of the pre norm, P, and with a gate per token and a layer norm b of
// the post norm (at V = 2 read where it is used).  A stage of the ring: R
// rows of dy, dh, y, a and, with a gate per token that has room (ring_gate),
// the gate.
template <typename Tx, typename Ta, int V, bool kVec, bool kNarrow, bool kLayer, bool kToken, int kBound>
__global__ void __launch_bounds__(kBound)
    block_norm_bwd_kernel(const BlockNormArgs p, const Split sp, const Partials pt, int stages, int ring_gate) {
  constexpr int R = 3 - V;  // rows at a time
  // Where a layer norm's sums leave no registers the post norm reads its
  // statistics again (16384 x 8192 in fp32 815 us, with them kept 908 us; 5003
  // x 4096 with a gate per token 68.7 and 69.2 us). Elsewhere they are kept
  // (32768 x 3584 283 us, read again 285 us).
  constexpr bool kReadAgain = kLayer && (kToken || (V == 2 && kBound == kThreads));
  extern __shared__ uint4 smem[];
  constexpr int kSums = kLayer ? 2 * R : R, kBuf = 32 * (V == 1 ? 2 * R : 2);
  __shared__ __align__(16) float bufs[8 * kBuf];
  const int D = p.D, group = static_cast<int>(threadIdx.x) / sp.threads;
  const int tid = static_cast<int>(threadIdx.x) - group * sp.threads, lane = tid & 31;  // of the group's
  const float inv_d = 1.f / static_cast<float>(D);
  const bool post = p.flags & kNormPost, pre = p.flags & kNormPre, sig = p.flags & kNormGateSigmoid;
  const bool has_a = p.a != nullptr;
  int col[V];
#pragma unroll
  for (int i = 0; i < V; ++i) col[i] = kVec ? 8 * (tid + i * sp.threads) : 8 * (V * tid + i);
  // groups of several warps are eight at most; barrier 0 is the CTA's
  const uint32_t mask = group_mask<kNarrow>(sp.threads);
  RowSum<kSums, kNarrow> sum{bufs + kBuf * (group & 7), mask, sp.threads, tid >> 5, group + 1, 0};
  for (int k = threadIdx.x; k < 8 * kBuf; k += blockDim.x) bufs[k] = 0.f;

  constexpr bool kKeepB = kToken && kLayer && V == 1;
  constexpr int plane = 32;
  const int my_warp = static_cast<int>(threadIdx.x) >> 5, all_warps = (static_cast<int>(blockDim.x) + 31) / 32;
  const bool own_post = !kToken && sp.G > 1;                    // P is of the unit's gate row
  const int weights = (own_post ? 2 : kKeepB ? 6 : 4) * V;      // planes that all groups share
  uint4* const w_pre = smem + (tid >> 5) * 32 * weights + lane;
  uint4* const b_post = w_pre + 4 * V * plane;
  uint4* const own = smem + (sp.threads + 31) / 32 * 32 * weights;
  uint4* const w_post = own_post ? own + my_warp * 2 * V * plane + (threadIdx.x & 31) : w_pre + 2 * V * plane;
  constexpr int kRowX = kRowPlanes<Tx, V, kVec>, kRowA = kRowPlanes<Ta, V, kVec>;
  constexpr int kDh = R * kRowX, kY = kDh + R * kRowA, kA = kY + R * kRowX, kG = kA + R * kRowA;
  const int row_g = p.dt_gate == kFp32 ? kRowPlanes<float, V, kVec> : kRowA;
  const int stage_step = (kG + (ring_gate ? R * row_g : 0)) * plane;
  uint4* const rings = own + (own_post ? all_warps * 2 * V * plane : 0);
  uint4* const ring = rings + my_warp * stages * stage_step + (threadIdx.x & 31);
  if (col[V - 1] + 8 > D || !p.dy)  // what is never fetched reads as zero
    for (int k = 0; k < stages * stage_step; k += plane) ring[k] = make_uint4(0, 0, 0, 0);
  // past the ring, the statistics of a stage's rows, a copy for each warp (or
  // group of part of one): {rstd of the post norm, of the pre norm, their
  // means}, of absent norms 1, 0, 0, 0
  float4* const my_stats = reinterpret_cast<float4*>(rings + all_warps * stages * stage_step) +
                           stages * R * (static_cast<int>(threadIdx.x) / (kNarrow ? sp.threads : 32));
  for (int k = lane; k < stages * R; k += (kNarrow ? sp.threads : 32)) my_stats[k] = make_float4(1.f, 0.f, 0.f, 0.f);
  __syncwarp(mask);

  // this group's units, and the rows that it takes one after another
  const long long worker = static_cast<long long>(blockIdx.x) * sp.groups + group;
  const long long workers = static_cast<long long>(gridDim.x) * sp.groups;
  const long long u0 = sp.units * worker / workers, u1 = sp.units * (worker + 1) / workers;
  const long long next = sp.S * R;  // from a unit's step to its next one
  struct Unit { long long row, end; };  // its first row, the end of its gate row
  auto unit = [&](long long u) {
    const long long g = u / sp.S, s = u - g * sp.S;
    return Unit{g * sp.rows + s * R, (g + 1) * sp.rows};
  };
  auto step_rows = [&](long long r, long long end) { return static_cast<int>(end - r < R ? end - r : R); };
  // lanes 4 q + k: row q's statistic k (0, 2: the post norm's)
  const bool stat_mine = lane < 4 * R && (lane & 1 ? pre : post) && (kLayer || !(lane & 2));
  auto fetch = [&](long long r0, int rows, int s_at) {
    uint4* at = ring + s_at * stage_step;
    if (stat_mine) {
      float* to = reinterpret_cast<float*>(&my_stats[s_at * R + (lane >> 2)]) + (lane & 3);
      if ((lane >> 2) < rows) cp_async4(to, p.stats + (lane & 3) * p.M + r0 + (lane >> 2));
      else *to = 0.f;
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (q >= rows) {  // a row that is not there adds nothing: zeros
        auto clear = [&](uint4* to, int planes) {
          for (int k = 0; k < planes; ++k) to[k * plane] = make_uint4(0, 0, 0, 0);
        };
        clear(at + q * kRowX * plane, kRowX);
        clear(at + (kDh + q * kRowA) * plane, kRowA);
        clear(at + (kY + q * kRowX) * plane, kRowX);
        clear(at + (kA + q * kRowA) * plane, kRowA);
        if (kToken && ring_gate) clear(at + (kG + q * row_g) * plane, row_g);
        break;
      }
      const long long r = r0 + q;
      if (p.dy) fetch_cols<Tx, kVec>(at + q * kRowX * plane, plane, static_cast<const Tx*>(p.dy), static_cast<const Tx*>(p.dy) + r * p.ld_dy, col, D);
      if (pre) {
        fetch_cols<Ta, kVec>(at + (kDh + q * kRowA) * plane, plane, static_cast<const Ta*>(p.dh), static_cast<const Ta*>(p.dh) + r * p.ld_dh, col, D);
        fetch_cols<Tx, kVec>(at + (kY + q * kRowX) * plane, plane, static_cast<const Tx*>(p.y), static_cast<const Tx*>(p.y) + r * p.ld_y, col, D);
      }
      if (has_a) fetch_cols<Ta, kVec>(at + (kA + q * kRowA) * plane, plane, static_cast<const Ta*>(p.a), static_cast<const Ta*>(p.a) + r * p.ld_a, col, D);
      if (kToken && ring_gate) {
        uint4* to = at + (kG + q * row_g) * plane;
        if (p.dt_gate == kFp32) fetch_cols<float, kVec>(to, plane, static_cast<const float*>(p.gate), static_cast<const float*>(p.gate) + r * p.ld_gate, col, D);
        else fetch_cols<Ta, kVec>(to, plane, static_cast<const Ta*>(p.gate), static_cast<const Ta*>(p.gate) + r * p.ld_gate, col, D);
      }
    }
  };
  long long ahead_unit = u0;  // what is fetched next
  Unit ahead = unit(u0);
  if (u0 == u1) ahead.end = ahead.row;
  auto fetch_next = [&](int s_at) {
    if (!kToken)  // (there a group has one unit at most)
      while (ahead_unit + 1 < u1 && ahead.row >= ahead.end) ahead = unit(++ahead_unit);
    if (ahead.row < ahead.end) {
      fetch(ahead.row, step_rows(ahead.row, ahead.end), s_at);
      ahead.row += next;
    }
    cp_commit();
  };
  for (int s = 0; s < stages - 1; ++s) fetch_next(s);

  Cols pre_w[V], pre_b[V], s1[V], s0[V];
#pragma unroll
  for (int i = 0; i < V; ++i) pre_w[i] = pre_b[i] = s1[i] = s0[i] = all_cols(0.f);
  // P: what dx is multiplied with before the post norm's own backward, scale
  // g w of gate row g (with a gate per token w alone)
  auto put_post = [&](long long g) {
    Cols P[V], e[V];
    weight_cols<kVec>(p.post_w, col, D, 1.f, P);
    if (sp.shared) gate_cols<Ta, kVec>(p, g, col, e);
    if (!kToken) {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          P[i].p[j] = mul2(P[i].p[j], sp.shared ? mul2(e[i].p[j], both(p.scale)) : both(p.scale));
    }
    put_cols(w_post, plane, P);
  };
  if (group == 0) {
    Cols w[V];
    weight_cols<kVec>(p.pre_w, col, D, 1.f, w);
    put_cols(w_pre, plane, w);
    if (kKeepB) {
      weight_cols<kVec>(p.post_b, col, D, 0.f, w);
      put_cols(b_post, plane, w);
    }
    if (!own_post) put_post(0);
  }
  __syncthreads();

  int stage = 0;
  for (long long u = u0; u < u1; ++u) {
    const long long g = u / sp.S;
    const Unit at_hand = unit(u);
    if (own_post) put_post(g);
    for (long long r = at_hand.row; r < at_hand.end; r += next) {
      const int rows = step_rows(r, at_hand.end);
      const uint4* at = ring + stage * stage_step;
      // (the warp has read the stage that is fetched into: its lanes met in
      // the row sums since)
      fetch_next(stage == 0 ? stages - 1 : stage - 1);
      cp_wait(stages - 1);
      __syncwarp(mask);
      float4 st[R];
#pragma unroll
      for (int q = 0; q < R; ++q) st[q] = my_stats[stage * R + q];

      // elements from the aligned bytes that row r + q was fetched from
      auto shift = [&](const void* base, long long ld, int q, auto t) {
        return shift_of<decltype(t), kVec>(static_cast<const decltype(t)*>(base) + (r + q) * ld);
      };
      Cols dx[R][V], hat[R][V];
      float2 c1[R], c2[R];
      // c1 = sum v hat, c2 = sum v over the row -> minus their means
      auto means = [&] {
        float c[kSums];
#pragma unroll
        for (int q = 0; q < R; ++q) {
          c[q] = sum2(c1[q]);
          if (kLayer) c[R * kLayer + q] = sum2(c2[q]);
        }
        sum(c);
#pragma unroll
        for (int q = 0; q < R; ++q) {
          c1[q] = both(c[q] * -inv_d);
          c2[q] = both(kLayer ? c[R * kLayer + q] * -inv_d : 0.f);
        }
      };
      if (pre) {
        Cols v[R][V];
#pragma unroll
        for (int q = 0; q < R; ++q) c1[q] = c2[q] = both(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const Cols w = weight_at(w_pre, plane, i);
#pragma unroll
          for (int q = 0; q < R; ++q) {
            v[q][i] = take8<Ta, kVec>(at + (kDh + q * kRowA) * plane, plane, i, shift(p.dh, p.ld_dh, q, Ta{}));
            hat[q][i] = take8<Tx, kVec>(at + (kY + q * kRowX) * plane, plane, i, shift(p.y, p.ld_y, q, Tx{}));
            normed<kLayer>(hat[q][i], st[q].w, st[q].y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float2 &d = v[q][i].p[j], &h = hat[q][i].p[j];
              pre_w[i].p[j] = fma2(d, h, pre_w[i].p[j]);
              if (kLayer) pre_b[i].p[j] = add2(pre_b[i].p[j], d);
              d = mul2(d, w.p[j]);
              c1[q] = fma2(d, h, c1[q]);
              if (kLayer) c2[q] = add2(c2[q], d);
            }
          }
        }
        means();
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dx[q][i] = take8<Tx, kVec>(at + q * kRowX * plane, plane, i, shift(p.dy, p.ld_dy, q, Tx{}));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float2 d = v[q][i].p[j];
              if (kLayer) d = add2(d, c2[q]);
              dx[q][i].p[j] = fma2(fma2(hat[q][i].p[j], c1[q], d), both(st[q].y), dx[q][i].p[j]);
            }
          }
      } else {
#pragma unroll
        for (int q = 0; q < R; ++q) take_cols<Tx, kVec>(at + q * kRowX * plane, plane, dx[q], shift(p.dy, p.ld_dy, q, Tx{}));
      }
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (q < rows) store_cols<Tx, kVec>(static_cast<Tx*>(p.dx) + (r + q) * p.ld_dx, col, D, dx[q], mask);
      if (has_a) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          c1[q] = c2[q] = both(0.f);
          // (the stage's until the lanes have met in the post norm's sums;
          // without that norm they are not used)
          if (kReadAgain) st[q] = stats_at(&my_stats[stage * R + q]);
        }
        Cols slopes[kToken && !kVec ? V : 1];  // (R is 1 there)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const Cols w = weight_at(w_post, plane, i);
#pragma unroll
          for (int q = 0; q < R; ++q) {
            hat[q][i] = take8<Ta, kVec>(at + (kA + q * kRowA) * plane, plane, i, shift(p.a, p.ld_a, q, Ta{}));
            if (post) normed<kLayer>(hat[q][i], st[q].z, st[q].x);
            if (kToken) {
              // the gate's own gradient, and dx behind the gate
              Cols e, slope;
              const uint4* from = at + (kG + q * row_g) * plane;
              if (!ring_gate) e = q < rows ? gate8<Ta, kVec>(p, r + q, col[i]) : all_cols(0.f);
              else if (p.dt_gate == kFp32) e = take8<float, kVec>(from, plane, i, shift(p.gate, p.ld_gate, q, float{}));
              else e = take8<Ta, kVec>(from, plane, i, shift(p.gate, p.ld_gate, q, Ta{}));
              gate_value(e, sig);
              if (kLayer) slope = kKeepB ? weight_at(b_post, plane, i) : weight8<kVec>(p.post_b, col[i], D, 0.f);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float2 &d = dx[q][i].p[j], &s = slope.p[j];
                s = kLayer ? fma2(hat[q][i].p[j], w.p[j], s) : mul2(hat[q][i].p[j], w.p[j]);
                d = mul2(d, both(p.scale));
                s = mul2(s, d);
                d = mul2(d, e.p[j]);
                if (sig) s = mul2(s, fma2(mul2(e.p[j], both(-1.f)), e.p[j], e.p[j]));
              }
              if constexpr (!kVec) {
                slopes[i] = slope;
              } else if (q < rows) {
                if (p.dt_gate == kFp32) store8(static_cast<float*>(p.dgate) + (r + q) * D, col[i], D, slope);
                else store8(static_cast<Ta*>(p.dgate) + (r + q) * D, col[i], D, slope);
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float2& d = dx[q][i].p[j];
              s1[i].p[j] = fma2(d, hat[q][i].p[j], s1[i].p[j]);
              if (kLayer) s0[i].p[j] = add2(s0[i].p[j], d);
              d = mul2(d, w.p[j]);
              c1[q] = fma2(d, hat[q][i].p[j], c1[q]);
              if (kLayer) c2[q] = add2(c2[q], d);
            }
          }
        }
        if constexpr (kToken && !kVec) {
          if (p.dt_gate == kFp32) store_cols<float, false>(static_cast<float*>(p.dgate) + r * D, col, D, slopes, mask);
          else store_cols<Ta, false>(static_cast<Ta*>(p.dgate) + r * D, col, D, slopes, mask);
        }
        if (post) {
          means();
#pragma unroll
          for (int q = 0; q < R; ++q)
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float2& d = dx[q][i].p[j];
                if (kLayer) d = add2(d, c2[q]);
                d = mul2(fma2(hat[q][i].p[j], c1[q], d), both(st[q].x));
              }
        }
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (q < rows) store_cols<Ta, kVec>(static_cast<Ta*>(p.da) + (r + q) * p.ld_da, col, D, dx[q], mask);
      }
      stage = stage + 1 < stages ? stage + 1 : 0;
    }
    if (kToken) break;
    // Several gate rows: the unit's sums of dx ahat and dx go to the weights'
    // gradients times scale g, to the gate's as scale (w s1 + b s0) g'.  With
    // one gate row both are left to the sum over the rows of partial sums.
    if (!kToken && sp.G > 1) {
      Cols e[V], w[V], t[V];
      gate_cols<Ta, kVec>(p, g, col, e);
      weight_cols<kVec>(p.post_w, col, D, 1.f, w);
      weight_cols<kVec>(p.post_b, col, D, 0.f, t);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[i].p[j] = mul2(fma2(w[i].p[j], s1[i].p[j], mul2(t[i].p[j], s0[i].p[j])), both(p.scale));
          if (sig) w[i].p[j] = mul2(w[i].p[j], fma2(mul2(e[i].p[j], both(-1.f)), e[i].p[j], e[i].p[j]));
        }
      store_cols<float, kVec>(sp.S > 1 ? pt.unit + u * D : static_cast<float*>(p.dgate) + g * D, col, D, w, mask);
      float* row = pt.row + worker * pt.n * D;
#pragma unroll
      for (int k = 0; k < (kLayer ? 2 : 1); ++k) {
        float* to = row + (k ? kPostB : kPostW) * D;
        weight_cols<kVec>(u == u0 ? nullptr : to, col, D, 0.f, t);
        Cols(&sums)[V] = k ? s0 : s1;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            t[i].p[j] = fma2(sums[i].p[j], mul2(e[i].p[j], both(p.scale)), t[i].p[j]);
            sums[i].p[j] = both(0.f);
          }
        store_cols<float, kVec>(to, col, D, t, mask);
      }
    }
  }
  if (!kToken && sp.G > 1) {
    float* row = pt.row + worker * pt.n * D;
    store_cols<float, kVec>(row + kPreW * D, col, D, pre_w, mask);
    if (kLayer) store_cols<float, kVec>(row + kPreB * D, col, D, pre_b, mask);
    if (u0 == u1) {  // no unit came
      store_cols<float, kVec>(row + kPostW * D, col, D, s1, mask);
      if (kLayer) store_cols<float, kVec>(row + kPostB * D, col, D, s0, mask);
    }
    return;
  }
  // the CTA's sums: its groups' added in order, through the shared memory
  // once every group is done with its own
  float* out = pt.row + static_cast<long long>(blockIdx.x) * pt.n * D;
  if (sp.groups == 1) {
    store_cols<float, kVec>(out + kPreW * D, col, D, pre_w, mask);
    store_cols<float, kVec>(out + kPostW * D, col, D, s1, mask);
    if (kLayer) {
      store_cols<float, kVec>(out + kPreB * D, col, D, pre_b, mask);
      store_cols<float, kVec>(out + kPostB * D, col, D, s0, mask);
    }
    return;
  }
  cp_wait(0);
  __syncthreads();
  // slots of thread t: its warp's planes together
  constexpr int kDump = (kLayer ? 4 : 2) * 2 * V;
  auto dump = [&](int t) { return smem + (t >> 5) * 32 * kDump + (t & 31); };
  uint4* const mine = dump(static_cast<int>(threadIdx.x));
  put_cols(mine + 2 * V * kPreW * plane, plane, pre_w);
  put_cols(mine + 2 * V * kPostW * plane, plane, s1);
  if (kLayer) {
    put_cols(mine + 2 * V * kPreB * plane, plane, pre_b);
    put_cols(mine + 2 * V * kPostB * plane, plane, s0);
  }
  __syncthreads();
  if (group > 0) return;
  for (int k = 0; k < (kLayer ? 4 : 2); ++k) {
    Cols t[V], o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = all_cols(0.f);
    for (int q = 0; q < sp.groups; ++q) {
      take_cols<float, true>(dump(q * sp.threads + tid) + 2 * V * k * plane, plane, o, 0);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) t[i].p[j] = add2(t[i].p[j], o[i].p[j]);
    }
    store_cols<float, kVec>(out + k * D, col, D, t, mask);
  }
}

// kBound: most threads of a CTA; less than kThreads for layer norms alone.
template <int V, bool kVec, bool kNarrow, int kBound = kThreads>
cudaError_t run_bwd(const BlockNormArgs& a, const Split& sp, const Partials& pt, cudaStream_t stream) {
  constexpr int R = 3 - V, kMost = (V == 2 ? kSmemWide : kSmem) + 1024;
  const bool layer_norm = a.flags & kNormLayer, token = a.gate && !sp.shared, own_post = sp.G > 1;
  const size_t plane = static_cast<size_t>(sp.threads * sp.groups + 31) / 32 * 512;  // of all threads
  const size_t fixed = static_cast<size_t>(sp.threads + 31) / 32 * 512 * (own_post ? 2 : token && layer_norm && V == 1 ? 6 : 4) * V +
                       (own_post ? 2 * V * plane : 0);
  const size_t own_stats = static_cast<size_t>(sp.threads) * sp.groups / (kNarrow ? sp.threads : 32) * R * 16;  // a stage's
  const size_t gate = token ? R * row_planes(a.dt_gate, V, kVec) * plane : 0;
  size_t stage = 2 * R * (row_planes(a.dt_x, V, kVec) + row_planes(a.dt_a, V, kVec)) * plane;
  const int ring_gate = token && fixed + stage + gate + own_stats <= kMost;
  if (ring_gate) stage += gate;
  // 100 KB ahead of the rows at hand, at least a stage; none where a stage
  // crowds memory by itself and another group works meanwhile (32768 x 3584
  // with an fp32 stream, 2 x 1, 86 KB, 374 us, 2 x 2 414 us)
  const bool crowded = stage > static_cast<size_t>(layer_norm ? 90 : 80) * 1024 && sp.groups > 1;
  const size_t ahead = crowded ? 0 : std::max<size_t>(100 * 1024 / stage, 1);
  const int stages = stages_for(stage + own_stats, std::min(kMost - fixed, (ahead + 1) * (stage + own_stats)));
  const size_t sums = sp.groups > 1 ? static_cast<size_t>(pt.n) * 2 * V * plane : 0;
  const size_t smem = std::max(fixed + (stage + own_stats) * stages, sums);
  if (smem > kMost) return cudaErrorInvalidValue;
  auto run = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    kernel<<<sp.ctas, sp.threads * sp.groups, smem, stream>>>(a, sp, pt, stages, ring_gate);
    return cudaGetLastError();
  };
  return by_types(a, [&](auto x, auto y) {
    using Tx = decltype(x);
    using Ta = decltype(y);
    if (layer_norm)
      return token ? run(block_norm_bwd_kernel<Tx, Ta, V, kVec, kNarrow, true, true, kBound>)
                   : run(block_norm_bwd_kernel<Tx, Ta, V, kVec, kNarrow, true, false, kBound>);
    if constexpr (kBound < kThreads)
      return cudaErrorInvalidValue;
    else
      return token ? run(block_norm_bwd_kernel<Tx, Ta, V, kVec, kNarrow, false, true, kBound>)
                   : run(block_norm_bwd_kernel<Tx, Ta, V, kVec, kNarrow, false, false, kBound>);
  });
}

// The variants, a translation unit each: eight columns and 16 columns a
// thread, and 16 of rows that are not whole 16-byte accesses, in groups of
// warps and of part of one.
cudaError_t run_bwd_8(const BlockNormArgs& a, const Split& sp, const Partials& pt, cudaStream_t stream);
cudaError_t run_bwd_16(const BlockNormArgs& a, const Split& sp, const Partials& pt, cudaStream_t stream);
cudaError_t run_bwd_16_layer(const BlockNormArgs& a, const Split& sp, const Partials& pt, cudaStream_t stream);
cudaError_t run_bwd_any(const BlockNormArgs& a, const Split& sp, const Partials& pt, cudaStream_t stream);
cudaError_t run_bwd_any_narrow(const BlockNormArgs& a, const Split& sp, const Partials& pt, cudaStream_t stream);

}  // namespace norm
}  // namespace ra
