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
#include "launch.hpp"
#include "w4a16_tile.hpp"
#include "wave.hpp"

namespace mxf {

namespace {

constexpr int kWaves = 8;        // of a forward workgroup
constexpr int kFinishGroups = 8;  // groups of 64 threads that share a sequence's slots

template <bool kBF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if (kBF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
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

// the sequences' bounds, held to [0, T] (no offsets: one sequence of all tokens)
__device__ __forceinline__ int64_t seg_begin(const RouteLossArgs& a, int s) {
  return a.seg_offsets ? min(max((int64_t)a.seg_offsets[s], (int64_t)0), a.T) : (s > 0 ? a.T : 0);
}

// the first sequence that ends past token t, by a whole wave
__device__ __forceinline__ int seg_of(const RouteLossArgs& a, int64_t t) {
  return a.seg_offsets ? first_segment(a.seg_offsets, a.S, t) : 0;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// One workgroup: tokens [tb blockIdx, tb (blockIdx + 1)), sequence after sequence. With one workgroup
// in the launch it writes the results itself.
template <bool kBF16, int V>
__global__ void __launch_bounds__(64 * kWaves) balance_kernel(RouteLossArgs a, int64_t tb) {
  constexpr int U = V <= 4 ? 4 : V <= 8 ? 2 : 1;  // tokens of a wave in flight
  __shared__ float red[kWaves][64 * V];
  __shared__ int32_t cnt[64 * V];
  __shared__ float zred[kWaves];
  __shared__ int32_t nred[kWaves];
  __shared__ double bred[kWaves];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int64_t t0 = (int64_t)blockIdx.x * tb, t1 = min(t0 + tb, a.T);
  const int E = a.E, topk = a.topk;
  const bool alone = gridDim.x == 1;
  const Slots slots = slots_at(a.workspace, gridDim.x, a.S, E);
  if (blockIdx.x == 0 && tid == 0) *slots.done = 0;
  for (int e = tid; e < 64 * V; e += 64 * kWaves) cnt[e] = 0;
  __syncthreads();

  double balance = 0.0, zsum = 0.0;  // of this thread / thread 0
  int64_t total = 0;
  int held = 0;
  int64_t covered = t0;
  auto uncovered = [&](int64_t to) {
    for (int64_t t = covered + tid; t < to; t += 64 * kWaves) a.lse[t] = -INFINITY;
    covered = max(covered, to);
  };

  for (int s = alone ? 0 : seg_of(a, t0); s < a.S; ++s) {
    const int64_t begin = seg_begin(a, s);
    if (begin >= t1 && !alone) break;
    const int64_t lo = max(begin, covered), hi = min(seg_begin(a, s + 1), t1);
    if (lo >= hi) {
      if (alone) {
        for (int e = tid; e < E; e += 64 * kWaves) {
          a.counts[(int64_t)s * E + e] = 0;
          a.prob_mean[(int64_t)s * E + e] = 0.0f;
        }
        if (tid == 0) a.tokens[s] = 0;
      }
      continue;
    }
    uncovered(lo);
    covered = hi;

    float P[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 0.0f;
    float z = 0.0f;
    int n = 0;
    for (int64_t t = lo + wave; t < hi; t += U * kWaves) {
      float x[U][V];
      bool use[U];
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t tu = t + u * kWaves;
        use[u] = tu < hi;
        const int64_t at = use[u] ? tu : t;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = lane + 64 * v;
          x[u][v] = e < E ? load_logit<kBF16>(a.logits, at * E + e) : -INFINITY;
        }
        id[u] = lane < topk ? a.topk_ids[at * topk + lane] : -1;
        if (a.token_mask && a.token_mask[at] == 0) use[u] = false;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float m = x[u][0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, x[u][v]);
        m = wave_max(m);
        if (m == -INFINITY) use[u] = false;  // no expert left
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          x[u][v] = __expf(x[u][v] - m);
          sum += x[u][v];
        }
        sum = wave_sum(sum);
        const float l = m + logf(sum);
        const int64_t tu = t + u * kWaves;
        if (lane == 0 && tu < hi) a.lse[tu] = use[u] ? l : -INFINITY;
        if (use[u]) {
          const float inv = 1.0f / sum;
#pragma unroll
          for (int v = 0; v < V; ++v) P[v] += x[u][v] * inv;
          z += l * l;
          ++n;
          if ((uint32_t)id[u] < (uint32_t)E) atomicAdd(&cnt[id[u]], 1);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) red[wave][lane + 64 * v] = P[v];
    if (lane == 0) {
      zred[wave] = z;
      nred[wave] = n;
    }
    __syncthreads();
    float zb = 0.0f;
    int nb = 0;
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
  }
  uncovered(t1);
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

// One workgroup per sequence and 64 experts: adds the sequence's slots; the last one to finish adds
// what all of them leave (each reads the others' values through the device-wide coherent point).
__global__ void __launch_bounds__(64 * kFinishGroups) balance_finish_kernel(RouteLossArgs a, int64_t tb, int64_t blocks) {
  __shared__ float pred[kFinishGroups][64];
  __shared__ int32_t cred[kFinishGroups][64], nred[kFinishGroups];
  __shared__ float zred[kFinishGroups];
  __shared__ double dred[2][kFinishGroups];
  __shared__ int64_t tred[2][kFinishGroups];
  __shared__ uint32_t last;
  const int tid = threadIdx.x, grp = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int E = a.E, EB = (E + 63) / 64;
  const Slots slots = slots_at(a.workspace, blocks, a.S, E);
  const int s = blockIdx.x / EB, eb = blockIdx.x % EB, e = 64 * eb + lane;
  const int64_t lo = seg_begin(a, s), hi = seg_begin(a, s + 1);
  const int64_t b0 = lo / tb, b1 = lo < hi ? (hi - 1) / tb + 1 : b0;
  float p = 0.0f, z = 0.0f;
  int32_t c = 0, n = 0;
#pragma unroll 4
  for (int64_t b = b0 + grp; b < b1; b += kFinishGroups) {
    const int64_t slot = b + s;
    if (e < E) {
      p += slots.p[slot * E + e];
      c += slots.c[slot * E + e];
    }
    z += slots.z[slot];
    n += slots.n[slot];
  }
  pred[grp][lane] = p;
  cred[grp][lane] = c;
  if (lane == 0) {
    zred[grp] = z;
    nred[grp] = n;
  }
  __syncthreads();
  if (grp == 0) {
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
    }
    const double bal = wave_sum_f64(e < E ? (double)c * (double)p * per * per : 0.0);
    if (lane == 0) {
      __hip_atomic_store(&slots.balance[blockIdx.x], bal, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (eb == 0) {
        __hip_atomic_store(&slots.zs[s], zd, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&a.tokens[s], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      last = __hip_atomic_fetch_add(slots.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1 == gridDim.x;
    }
  }
  __syncthreads();
  if (!last) return;
  double bal = 0.0, zd = 0.0;
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

// d logits: one wave per token
template <bool kBF16, int V>
__global__ void __launch_bounds__(256) route_backward_kernel(RouteLossArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E, topk = a.topk;
  float x[V];
  const bool losses = a.dlosses != nullptr;
  float l = -INFINITY;
  if (losses) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + 64 * v;
      x[v] = e < E ? load_logit<kBF16>(a.logits, t * E + e) : -INFINITY;
    }
    l = a.lse[t];
  }
  float g = 0.0f, dg = 0.0f;
  int id = -1;
  if (a.dgates && lane < topk) {
    g = a.gates[t * topk + lane];
    dg = a.dgates[t * topk + lane];
    id = a.topk_ids[t * topk + lane];
  }
  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = 0.0f;
  if (l != -INFINITY) {
    const int s = seg_of(a, t);
    if (s < a.S) {
      const float n = (float)a.tokens[s], total = (float)a.tokens[a.S], held = (float)a.tokens[a.S + 1];
      const float kb = a.dlosses[0] * ((float)E / ((float)topk * held)) / n, kz = a.dlosses[1] * 2.0f * l / total;
      // p from the row itself: lse holds log(sum exp(x - max)) only as far as the maximum's size leaves it bits
      float m = x[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
      m = wave_max(m);
      float c[V], dot = 0.0f, sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane + 64 * v;
        c[v] = e < E ? (float)a.counts[(int64_t)s * E + e] / n : 0.0f;
        x[v] = __expf(x[v] - m);
        sum += x[v];
        dot += x[v] * c[v];
      }
      const float inv = 1.0f / wave_sum(sum);
      dot = wave_sum(dot) * inv;
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = x[v] * inv * (kb * (c[v] - dot) + kz);
    }
  }
  if (a.dgates) {
    const float mine = g * (dg - wave_sum(g * dg));
    for (int j = 0; j < topk; ++j) {
      const int ij = __builtin_amdgcn_readlane(id, j);
      const float dj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), j));
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (ij == lane + 64 * v) d[v] += dj;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    if (e < E) {
      if (kBF16) static_cast<__bf16*>(a.dlogits)[t * E + e] = (__bf16)d[v];
      else static_cast<float*>(a.dlogits)[t * E + e] = d[v];
    }
  }
}

// Tokens of a forward workgroup: at least 64, and at most 1024 workgroups. At most 64 tokens are one
// workgroup that writes the results itself (no second launch).
int64_t tokens_per_block(int64_t T) { return cdiv(max(T, (int64_t)1), 1024) > 64 ? cdiv(T, 1024) : 64; }

template <bool kBF16>
void launch_forward(const RouteLossArgs& a, int64_t tb, unsigned blocks, hipStream_t stream) {
  const dim3 threads(64 * kWaves);
  if (a.E <= 64) balance_kernel<kBF16, 1><<<blocks, threads, 0, stream>>>(a, tb);
  else if (a.E <= 128) balance_kernel<kBF16, 2><<<blocks, threads, 0, stream>>>(a, tb);
  else if (a.E <= 256) balance_kernel<kBF16, 4><<<blocks, threads, 0, stream>>>(a, tb);
  else if (a.E <= 512) balance_kernel<kBF16, 8><<<blocks, threads, 0, stream>>>(a, tb);
  else balance_kernel<kBF16, 16><<<blocks, threads, 0, stream>>>(a, tb);
}

template <bool kBF16>
void launch_backward(const RouteLossArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(a.T, 4)), threads(256);
  if (a.E <= 64) route_backward_kernel<kBF16, 1><<<grid, threads, 0, stream>>>(a);
  else if (a.E <= 128) route_backward_kernel<kBF16, 2><<<grid, threads, 0, stream>>>(a);
  else if (a.E <= 256) route_backward_kernel<kBF16, 4><<<grid, threads, 0, stream>>>(a);
  else if (a.E <= 512) route_backward_kernel<kBF16, 8><<<grid, threads, 0, stream>>>(a);
  else route_backward_kernel<kBF16, 16><<<grid, threads, 0, stream>>>(a);
}

}  // namespace

size_t route_loss_workspace(int64_t T, int64_t E, int64_t S) {
  const int64_t blocks = cdiv(max(T, (int64_t)1), tokens_per_block(T));
  const Slots s = slots_at(nullptr, blocks, S, E);
  return reinterpret_cast<size_t>(s.done) + sizeof(uint32_t);
}

int launch_route_loss(const RouteLossArgs& a, bool bf16, hipStream_t stream) {
  const int64_t tb = tokens_per_block(a.T), blocks = cdiv(max(a.T, (int64_t)1), tb);
  if (bf16) launch_forward<true>(a, tb, (unsigned)blocks, stream);
  else launch_forward<false>(a, tb, (unsigned)blocks, stream);
  if (blocks > 1)
    balance_finish_kernel<<<(unsigned)(a.S * cdiv(a.E, 64)), 64 * kFinishGroups, 0, stream>>>(a, tb, blocks);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_route_backward(const RouteLossArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) launch_backward<true>(a, stream);
  else launch_backward<false>(a, stream);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace mxf
