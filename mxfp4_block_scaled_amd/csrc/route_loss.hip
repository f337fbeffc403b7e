// The load-balance and z losses of a router with their per-expert counts, and the router's gradient.
//
// With p = softmax(logits) over all experts, lse its logarithm of the sum, sequences s of n_s tokens
// that count, c_si pairs and P_si = mean over s of p_i:
//   balance = 1/S' sum_s E / (topk n_s) sum_i c_si P_si,   z = 1/n sum_t lse_t^2
//   d logits_ti = g_b E / (S' topk n_s^2) p_i (c_si - sum_j p_j c_sj) + g_z 2/n lse p_i
//                 + sum_{j: id_j = i} gate_j (dgate_j - sum_k gate_k dgate_k)
// (S' sequences that hold a token, n tokens in all; counts have no gradient.)
//
// A wave holds a token's logits, lane l experts l + 64 v, so rows are read once and whole lines at a
// time whatever E is. Sums over tokens are kept apart by workgroup and sequence (slot = workgroup +
// sequence: both ascend along the tokens, so each pair that meets has a slot of its own) and added
// in a fixed order by a second launch: no floating-point atomics, the same result every time.
//
// Latency bounds all but the largest calls: 16384 x 256 fp32 in 16 sequences 11.9 + 6.4 to 7.7 us
// forward and 12.3 backward, of which the bytes are 3.5 and 7; 64 tokens 7.8 and 3.4.
#include "launch.hpp"
#include "w4a16_tile.hpp"
#include "wave.hpp"

namespace mxf {

namespace {

constexpr int kWaves = 8;         // of a forward workgroup
constexpr int kFinishGroups = 8;  // groups of 64 threads that share a sequence's slots
constexpr int kFinishLoads = 8;   // slots of a group in flight
constexpr int64_t kMostFinish = 512;  // workgroups

// Rows [row, row + U) of an [T][E] matrix as a range-checked resource: rows past T read as zeros. A row's or column's
// step goes into the vector offset: the check covers that for any size, a scalar offset only up to the resource's.
template <int U>
__device__ __forceinline__ buf_rsrc rows_of(const void* p, int64_t row, int64_t T, int E, int bytes) {
  const int64_t left = min((int64_t)U, T - row);
  return make_rsrc(static_cast<const char*>(p) + (left > 0 ? row * E * bytes : 0), left > 0 ? (uint32_t)(left * E * bytes) : 0);
}

// value e (a lane's) of row u
template <bool kBF16>
__device__ __forceinline__ float load_logit(buf_rsrc r, int u, int E, int e) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int at = u * E + e;
  if (kBF16) return __uint_as_float((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, 2 * at, 0, 0) << 16);
  return __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, 4 * at, 0, 0));
#else
  return 0.0f;
#endif
}

struct Slots {  // the workspace
  float* p;
  int32_t* c;
  float* z;
  int32_t* n;
  double* balance;  // [S][cdiv(E, 64)]
  double* zs;       // [S]
  uint32_t* done;
};

__host__ __device__ inline Slots slots_at(void* ws, int64_t blocks, int64_t S, int64_t E) {
  const int64_t n = blocks + S;
  Slots s;
  s.balance = static_cast<double*>(ws);
  s.zs = s.balance + S * cdiv(E, 64);
  s.p = reinterpret_cast<float*>(s.zs + S);
  s.c = reinterpret_cast<int32_t*>(s.p + n * E);
  s.z = reinterpret_cast<float*>(s.c + n * E);
  s.n = reinterpret_cast<int32_t*>(s.z + n);
  s.done = reinterpret_cast<uint32_t*>(s.n + n);
  return s;
}

// The sequences' bounds, held to [0, T] (no offsets: one sequence of all tokens). Up to 64 sequences' are
// read once, one a lane, so that walking them needs no further loads. Used by whole waves.
struct Bounds {
  const int32_t* off;
  int64_t T;
  int S, begins, ends;

  __device__ __forceinline__ explicit Bounds(const RouteLossArgs& a) : off(a.seg_offsets), T(a.T), S(a.S), begins(0), ends(0) {
    if (off && S <= 64) {
      const int i = min((int)(threadIdx.x & 63), S - 1);
      begins = off[i];
      ends = off[i + 1];
    }
  }
  __device__ __forceinline__ int64_t held(int v) const { return min(max((int64_t)v, (int64_t)0), T); }
  __device__ __forceinline__ int64_t begin(int s) const {
    return !off ? 0 : held(S <= 64 ? __builtin_amdgcn_readlane(begins, s) : off[s]);
  }
  __device__ __forceinline__ int64_t end(int s) const {
    return !off ? T : held(S <= 64 ? __builtin_amdgcn_readlane(ends, s) : off[s + 1]);
  }
  // the first sequence that ends past token t
  __device__ __forceinline__ int of(int64_t t) const {
    if (!off) return 0;
    if (S > 64) return first_segment(off, S, t);
    return __popcll(__ballot((int)(threadIdx.x & 63) < S && (int64_t)ends <= t));
  }
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// One workgroup: tokens [tb blockIdx, tb (blockIdx + 1)), 8 TW at a time, TW a wave. All loads go out
// first and the tokens' probabilities are formed without regard to sequences; then the workgroup walks the
// sequences that meet its tokens and keeps each one's sums in registers until it ends. Alone
// it writes the results itself.
template <bool kBF16, int V, int TW>
__global__ void __launch_bounds__(64 * kWaves) balance_kernel(RouteLossArgs a, int64_t tb, bool alone) {
  static_assert(TW <= 8, "8 lanes a token for its picks");
  __shared__ float red[kWaves][64 * V];
  __shared__ int32_t cnt[64 * V];
  __shared__ float zred[kWaves];
  __shared__ int32_t nred[kWaves];
  __shared__ double bred[kWaves];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int64_t t0 = (int64_t)blockIdx.x * tb, t1 = min(t0 + tb, a.T);
  const int E = a.E, topk = a.topk;
  const Slots slots = slots_at(a.workspace, gridDim.x, a.S, E);
  if (!alone && blockIdx.x == 0 && tid == 0) *slots.done = 0;

  double balance = 0.0, zsum = 0.0;  // of this thread / thread 0
  int64_t total = 0;
  int held = 0;
  const Bounds seg(a);
  int s = -1;
  float P[V] = {}, z = 0.0f;  // of this wave, for the sequence s
  int n = 0;

  // the end of sequence s here: the waves' sums to its slot
  auto flush = [&]() {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      red[wave][lane + 64 * v] = P[v];
      P[v] = 0.0f;
    }
    if (lane == 0) {
      zred[wave] = z;
      nred[wave] = n;
    }
    z = 0.0f;
    n = 0;
    __syncthreads();
    float zb = 0.0f;
    int nb = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      zb += zred[w];
      nb += nred[w];
    }
    const int64_t slot = alone ? s : (int64_t)blockIdx.x + s;
    const float per = nb > 0 ? 1.0f / (float)nb : 0.0f;
    for (int e = tid; e < E; e += 64 * kWaves) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) p += red[w][e];
      const int32_t c = cnt[e];
      cnt[e] = 0;
      if (alone) {
        a.counts[slot * E + e] = c;
        a.prob_mean[slot * E + e] = nb > 0 ? p / (float)nb : 0.0f;
        balance += (double)c * (double)p * (double)per * (double)per;
      } else {
        slots.p[slot * E + e] = p;
        slots.c[slot * E + e] = c;
      }
    }
    if (tid == 0) {
      if (alone) {
        a.tokens[s] = nb;
        zsum += zb;
      } else {
        slots.z[slot] = zb;
        slots.n[slot] = nb;
      }
    }
    total += nb;
    held += nb > 0;
    __syncthreads();
  };

  for (int64_t base = t0; base < t1 || (alone && base == t0); base += kWaves * TW) {
    const int64_t tw = base + wave * TW, hi = min(base + kWaves * TW, t1);  // the wave's first token
    float x[TW][V], l[TW];
    int id = -1;
    bool masked = false;
    const buf_rsrc rx = rows_of<TW>(a.logits, tw, a.T, E, kBF16 ? 2 : 4);
#pragma unroll
    for (int u = 0; u < TW; ++u)
#pragma unroll
      for (int v = 0; v < V; ++v)  // past the experts or tokens: some value, left out below
        x[u][v] = load_logit<kBF16>(rx, u, E, lane + 64 * v);
    if (a.T > 0) {
      id = a.topk_ids[min(tw + (lane >> 3), a.T - 1) * topk + min(lane & 7, topk - 1)];
      if (a.token_mask) masked = a.token_mask[min(tw + (lane & 7), a.T - 1)] == 0;
    }
    if (base == t0) {
      for (int e = tid; e < 64 * V; e += 64 * kWaves) cnt[e] = 0;
      if (s < 0) s = alone ? 0 : seg.of(t0);
      __syncthreads();
    }
    uint32_t use = 0;  // bit u: token tw + u is here and some of its experts are left
    const uint32_t out = (uint32_t)__ballot(masked);
#pragma unroll
    for (int u = 0; u < TW; ++u) {
      float m = -INFINITY;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (lane + 64 * v >= E) x[u][v] = -INFINITY;
        m = fmaxf(m, x[u][v]);
      }
      m = fmaxf(wave_max(m), -3.402823466e38f);  // so that a row of -inf alone has the sum 0, one with NaN the sum NaN
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[u][v] = __expf(x[u][v] - m);
        sum += x[u][v];
      }
      sum = wave_sum(sum);
      l[u] = m + logf(sum);
      const float inv = 1.0f / sum;
#pragma unroll
      for (int v = 0; v < V; ++v) x[u][v] *= inv;
      if (tw + u < hi && sum != 0.0f && !(out >> u & 1)) use |= 1u << u;
    }

    uint32_t counted = 0;
    while (s < a.S) {
      const int64_t from = seg.begin(s), to = seg.end(s);
      if (from >= hi && !(alone && hi >= t1)) break;  // it begins later
#pragma unroll
      for (int u = 0; u < TW; ++u) {
        if ((use >> u & 1) && tw + u >= from && tw + u < to) {
          counted |= 1u << u;
#pragma unroll
          for (int v = 0; v < V; ++v) P[v] += x[u][v];
          z += l[u] * l[u];
          ++n;
        }
      }
      const int64_t mine = tw + (lane >> 3);
      if ((lane >> 3) < TW && (lane & 7) < topk && (use >> (lane >> 3) & 1) && mine >= from && mine < to &&
          (uint32_t)id < (uint32_t)E)
        atomicAdd(&cnt[id], 1);
      const bool more = to > hi;            // it goes on behind these tokens
      if (more && hi < t1) break;           // in this workgroup
      if (from < to || alone) {
        __syncthreads();
        flush();
      }
      if (more) break;
      s = from < to || alone || a.S <= 64 ? s + 1 : max(s + 1, seg.of(to));  // over a run of empty ones at once
    }
    float mine = -INFINITY;
#pragma unroll
    for (int u = 0; u < TW; ++u)
      if (lane == u && (counted >> u & 1)) mine = l[u];
    if (lane < TW && tw + lane < hi) a.lse[tw + lane] = mine;
  }
  if (alone) {
    balance = wave_sum_f64(balance);
    if (lane == 0) bred[wave] = balance;
    __syncthreads();
    if (tid == 0) {
      double b = 0.0;
      for (int w = 0; w < kWaves; ++w) b += bred[w];
      a.losses[0] = (float)(b * E / ((double)topk * max(held, 1)));
      a.losses[1] = (float)(zsum / (double)max(total, (int64_t)1));
      a.tokens[a.S] = (int32_t)total;
      a.tokens[a.S + 1] = held;
    }
  }
}

// A workgroup takes a sequence and 64 experts at a time and adds its slots; the last one to finish adds
// what all of them leave (each reads the others' values through the device-wide coherent point). Few of them, as each
// adds a turn of 20 ns at the shared counter: 16384 x 256 in 1000 sequences, 4000 pairs of sequence and experts, 98 us
// for both launches with a workgroup a pair, 49, 42 and 49 in 1024, 512 and 256 of them.
__global__ void __launch_bounds__(64 * kFinishGroups) balance_finish_kernel(RouteLossArgs a, int64_t tb, int64_t blocks) {
  __shared__ float pred[kFinishGroups][64];
  __shared__ int32_t cred[kFinishGroups][64], nred[kFinishGroups];
  __shared__ float zred[kFinishGroups];
  __shared__ double dred[2][kFinishGroups];
  __shared__ int64_t tred[2][kFinishGroups];
  __shared__ uint32_t last;
  const int tid = threadIdx.x, grp = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int E = a.E, EB = (E + 63) / 64, items = a.S * EB;
  const Slots slots = slots_at(a.workspace, blocks, a.S, E);
  const Bounds seg(a);
  double bal = 0.0;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int s = it / EB, eb = it % EB, e = 64 * eb + lane;
    const int64_t lo = seg.begin(s), hi = seg.end(s);
    const int64_t b0 = lo / tb, b1 = lo < hi ? (hi - 1) / tb + 1 : b0;
    float p = 0.0f, z = 0.0f;
    int32_t c = 0, n = 0;
    for (int64_t b = b0 + grp; b < b1; b += kFinishLoads * kFinishGroups) {
      float ps[kFinishLoads], zs[kFinishLoads];
      int32_t cs[kFinishLoads], ns[kFinishLoads];
#pragma unroll
      for (int i = 0; i < kFinishLoads; ++i) {
        const int64_t slot = min(b + i * kFinishGroups, b1 - 1) + s;
        ps[i] = slots.p[slot * E + min(e, E - 1)];
        cs[i] = slots.c[slot * E + min(e, E - 1)];
        zs[i] = slots.z[slot];
        ns[i] = slots.n[slot];
      }
#pragma unroll
      for (int i = 0; i < kFinishLoads; ++i) {
        const bool in = b + i * kFinishGroups < b1;
        p += in ? ps[i] : 0.0f;
        c += in ? cs[i] : 0;
        z += in ? zs[i] : 0.0f;
        n += in ? ns[i] : 0;
      }
    }
    if (it >= (int)gridDim.x) __syncthreads();  // the last pair's sums are read
    pred[grp][lane] = p;
    cred[grp][lane] = c;
    if (lane == 0) {
      zred[grp] = z;
      nred[grp] = n;
    }
    __syncthreads();
    if (grp != 0) continue;
    p = 0.0f;
    c = n = 0;
    double zd = 0.0;
#pragma unroll
    for (int g = 0; g < kFinishGroups; ++g) {
      p += pred[g][lane];
      c += cred[g][lane];
      n += nred[g];
      zd += zred[g];
    }
    const double per = n > 0 ? 1.0 / (double)n : 0.0;
    if (e < E) {
      a.counts[(int64_t)s * E + e] = c;
      a.prob_mean[(int64_t)s * E + e] = n > 0 ? p / (float)n : 0.0f;
      bal += (double)c * (double)p * per * per;
    }
    if (lane == 0 && eb == 0) {
      __hip_atomic_store(&slots.zs[s], zd, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&a.tokens[s], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (grp == 0) {
    bal = wave_sum_f64(bal);
    if (lane == 0) {
      __hip_atomic_store(&slots.balance[blockIdx.x], bal, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(slots.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1 == gridDim.x;
    }
  }
  __syncthreads();
  if (!last) return;
  bal = 0.0;
  double zd = 0.0;
  int64_t total = 0, held = 0;
  for (int64_t i = tid; i < (int64_t)gridDim.x; i += 64 * kFinishGroups)
    bal += __hip_atomic_load(&slots.balance[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int64_t i = tid; i < a.S; i += 64 * kFinishGroups) {
    zd += __hip_atomic_load(&slots.zs[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int32_t m = __hip_atomic_load(&a.tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    total += m;
    held += m > 0;
  }
  bal = wave_sum_f64(bal);
  zd = wave_sum_f64(zd);
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    total += __shfl_xor(total, d);
    held += __shfl_xor(held, d);
  }
  if (lane == 0) {
    dred[0][grp] = bal;
    dred[1][grp] = zd;
    tred[0][grp] = total;
    tred[1][grp] = held;
  }
  __syncthreads();
  if (tid == 0) {
    bal = zd = 0.0;
    total = held = 0;
    for (int g = 0; g < kFinishGroups; ++g) {
      bal += dred[0][g];
      zd += dred[1][g];
      total += tred[0][g];
      held += tred[1][g];
    }
    a.losses[0] = (float)(bal * E / ((double)a.topk * (double)max(held, (int64_t)1)));
    a.losses[1] = (float)(zd / (double)max(total, (int64_t)1));
    a.tokens[a.S] = (int32_t)total;
    a.tokens[a.S + 1] = (int32_t)held;
  }
}

// d logits: one token a wave (two or four took 14 us where this takes 12, 16384 x 256 fp32: more waves have
// the loads' and the stores' turns beside each other). All loads that need no other go out first.
template <bool kBF16, int V>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteLossArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E, topk = a.topk;
  const bool losses = a.dlosses != nullptr;
  float x[V], d[V], l = -INFINITY, g = 0.0f, dg = 0.0f;
  int id = -1;
  if (losses) {
    const buf_rsrc rx = rows_of<1>(a.logits, t, a.T, E, kBF16 ? 2 : 4);
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = load_logit<kBF16>(rx, 0, E, lane + 64 * v);
    l = a.lse[t];
  }
  if (a.dgates) {  // lanes past topk: zeros, out of the row's range
    g = load_logit<false>(rows_of<1>(a.gates, t, a.T, topk, 4), 0, 0, lane);
    dg = load_logit<false>(rows_of<1>(a.dgates, t, a.T, topk, 4), 0, 0, lane);
    id = (int)__float_as_uint(load_logit<false>(rows_of<1>(a.topk_ids, t, a.T, topk, 4), 0, 0, lane));
  }
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = 0.0f;
  if (losses) {
    const Bounds seg(a);
    const float gb = a.dlosses[0], gz = a.dlosses[1];
    const float total = (float)a.tokens[a.S], held = (float)a.tokens[a.S + 1];
    const int s = min(seg.of(t), a.S - 1);
    const float n = (float)a.tokens[s];
    const buf_rsrc rc = rows_of<1>(a.counts, s, a.S, E, 4);
    float c[V], m = -INFINITY, sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = (float)(int)__float_as_uint(load_logit<false>(rc, 0, 0, lane + 64 * v));
    // p from the row itself: lse holds log(sum exp(x - max)) only as far as the maximum's size leaves it bits
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (lane + 64 * v >= E) x[v] = -INFINITY;
      m = fmaxf(m, x[v]);
    }
    m = wave_max(m);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = __expf(x[v] - m);
      sum += x[v];
    }
    const float inv = 1.0f / wave_sum(sum);
#pragma unroll
    for (int v = 0; v < V; ++v) dot += x[v] * c[v];
    dot = wave_sum(dot) * inv;
    if (l != -INFINITY) {  // the token counts
      const float kb = gb * ((float)E / ((float)topk * held)) / (n * n), kz = gz * 2.0f * l / total;
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = x[v] * inv * (kb * (c[v] - dot) + kz);
    }
  }
  if (a.dgates) {
    float dot = g * dg;  // over the first 8 lanes
    dot += dpp_move<0xB1>(dot);
    dot += dpp_move<0x4E>(dot);
    dot += dpp_move<0x141>(dot);
    const float mine = g * (dg - dot);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= topk) break;
      const int ij = __builtin_amdgcn_readlane(id, j);
      const float dj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), j));
      const float add = lane == (ij & 63) ? dj : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (ij >> 6 == v) d[v] += add;  // the whole wave takes one of these
    }
  }
  const buf_rsrc ro = rows_of<1>(a.dlogits, t, a.T, E, kBF16 ? 2 : 4);
#pragma unroll
  for (int v = 0; v < V; ++v) {  // lanes past the experts are out of the row's range
#if defined(__HIP_DEVICE_COMPILE__)
    if (kBF16) __builtin_amdgcn_raw_buffer_store_b16((short)bf16x2_bits(d[v], 0.0f), ro, 2 * (lane + 64 * v), 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32((int)__float_as_uint(d[v]), ro, 4 * (lane + 64 * v), 0, 0);
#endif
  }
}

// How the forward pass deals out T tokens: at most 64 in one or two sequences are one workgroup that writes the
// results itself, one sequence after the other (64 x 256 in 1, 2, 4 and 64 sequences: 8.0, 9.3, 11.8 and 85 us,
// with the second launch 10.0, 10.1, 10.5 and 29); else 2, 4 or 8 a wave, so that few tokens are many workgroups but a
// sequence has few slots to add (one sequence of 16384 tokens of 256 experts: 19 us in 256 workgroups, 26 in 512, 40 in
// 1024), and at most 512 workgroups.
constexpr int64_t kMostAlone = 2;
struct Deal {
  int tw;
  int64_t tb, blocks;
  bool alone;
};
Deal deal_of(int64_t T, int64_t S) {
  if (T <= 64 && S <= kMostAlone) return {8, 64, 1, true};
  const int tw = T <= 4096 ? 2 : T <= 8192 ? 4 : 8;
  const int64_t one = kWaves * tw, tb = one * max(cdiv(cdiv(T, one), 512), (int64_t)1);
  return {tw, tb, max(cdiv(T, tb), (int64_t)1), false};
}

template <bool kBF16, int V>
void launch_forward(const RouteLossArgs& a, const Deal& d, hipStream_t stream) {
  if (d.tw == 2) balance_kernel<kBF16, V, 2><<<(unsigned)d.blocks, 64 * kWaves, 0, stream>>>(a, d.tb, d.alone);
  else if (d.tw == 4) balance_kernel<kBF16, V, 4><<<(unsigned)d.blocks, 64 * kWaves, 0, stream>>>(a, d.tb, d.alone);
  else balance_kernel<kBF16, V, 8><<<(unsigned)d.blocks, 64 * kWaves, 0, stream>>>(a, d.tb, d.alone);
}

template <bool kBF16, int V>
void launch_backward(const RouteLossArgs& a, hipStream_t stream) {
  route_backward_kernel<kBF16, V><<<(unsigned)cdiv(a.T, 4), 256, 0, stream>>>(a);
}

template <bool kBF16>
void launch_both(const RouteLossArgs& a, bool backward, hipStream_t stream) {
  const Deal d = deal_of(a.T, a.S);
  if (a.E <= 64) backward ? launch_backward<kBF16, 1>(a, stream) : launch_forward<kBF16, 1>(a, d, stream);
  else if (a.E <= 128) backward ? launch_backward<kBF16, 2>(a, stream) : launch_forward<kBF16, 2>(a, d, stream);
  else if (a.E <= 256) backward ? launch_backward<kBF16, 4>(a, stream) : launch_forward<kBF16, 4>(a, d, stream);
  else if (a.E <= 512) backward ? launch_backward<kBF16, 8>(a, stream) : launch_forward<kBF16, 8>(a, d, stream);
  else backward ? launch_backward<kBF16, 16>(a, stream) : launch_forward<kBF16, 16>(a, d, stream);
}

}  // namespace

size_t route_loss_workspace(int64_t T, int64_t E, int64_t S) {
  const Deal d = deal_of(T, S);
  if (d.alone) return 0;
  return reinterpret_cast<size_t>(slots_at(nullptr, d.blocks, S, E).done) + sizeof(uint32_t);
}

int launch_route_loss(const RouteLossArgs& a, bool bf16, hipStream_t stream) {
  bf16 ? launch_both<true>(a, false, stream) : launch_both<false>(a, false, stream);
  const Deal d = deal_of(a.T, a.S);
  if (!d.alone)
    balance_finish_kernel<<<(unsigned)min(a.S * cdiv(a.E, 64), kMostFinish), 64 * kFinishGroups, 0, stream>>>(a, d.tb, d.blocks);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_route_backward(const RouteLossArgs& a, bool bf16, hipStream_t stream) {
  bf16 ? launch_both<true>(a, true, stream) : launch_both<false>(a, true, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
