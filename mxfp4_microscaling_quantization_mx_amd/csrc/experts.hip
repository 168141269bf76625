// The router of an expert layer for gfx950, and the sort of its slots by expert.
//
// Router.  Each token's `top` experts are those of its largest logits, largest
// first (ties to the lowest index, NaN above every number), and their weights
// come from the logits l:
//   softmax   w_j = scale e^(l_j - m) / sum e^(l_i - m), over the chosen
//             (renormalized) or over all experts, m the largest of them
//   sigmoid   w_j = scale s(l_j), or renormalized scale s(l_j) / sum s(l_i) over
//             the chosen, with s(l) = e^min(l, 0) / (1 + e^-|l|); the quotient
//             takes e^(min(l, 0) - max) so that it holds where every s underflows
// Where the largest logit of the set is -Inf the weights are 0.  The gradient
// recomputes them from the logits (p_j = w_j / scale, D = sum p_i dw_i):
//   softmax over the chosen  dl_j = scale p_j (dw_j - D)
//   softmax over all         dl_e = scale p_e ([e chosen] dw_e - D)
//   sigmoid                  dl_j = scale dw_j s_j (1 - s_j), renormalized
//                            dl_j = scale p_j (1 - s_j) (dw_j - D)
//
// A row is held by a group of G lanes, V consecutive logits each, as order-
// preserving 32-bit keys; a choice is a maximum over the group (DPP), and a
// ballot that names the lowest lane holding it.  Lane j then has the j-th chosen
// logit and the softmax runs across the group.  Little is read (1 MB for 16384
// tokens of 32 experts): the launch and the latency of one row bound it, 3.4-4 us for
// 16 tokens of 128 experts, 16384 of 32 and its backward pass alike (7.5 with the
// call); 16384 of 256 experts, top 8, 10.1 us, of 1024 25.7 (1.3 TB/s: eight
// reductions over 64 lanes).
//
// Sort.  A stable counting sort of the slots (token t, choice j) at 4 t + j and
// the like: chunks of 4096 slots, 16 waves of 4 rounds of 64.  In a round every
// lane finds the lanes of its expert with one ballot per bit of the expert's
// number, so its rank is a bit count and the lowest such lane alone moves the
// wave's counter: no atomics in the ranks, the same order on every run.  One
// workgroup takes up to one chunk in a single launch; more chunks are first
// counted by one launch and placed by another, each workgroup of which adds up the
// counts of all chunks in LDS (past SORT_DIRECT chunks a launch between them turns the
// counts into running sums).  64 slots 3.3 us (7.9 with the call), 65536 slots of
// 32 experts 4.2 + 5.6-6.4 us, each of the two its launch and two trips to memory;
// 262144 of 128 experts 13.2 us, a million of 256 20.6 (three launches).
#include "mx_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

// ---------------------------------------------------------------- router
// A float32 as an unsigned number of the same order: -Inf lowest (but above 0,
// which marks an absent one), the zeros equal, NaN highest.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return x != x ? 0xFFFFFFFFu : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// e^x for x <= 0 within 2 ulp: x log2 e in two parts, the second of which moves
// the result by less than 2^-16 of itself.  Below 2^-126 it is 0, so that a weight may err
// by that over its sum, which is 1/2 (sigmoid) or more; NaN stays.
__device__ __forceinline__ float exp_neg(float x) {
  const float c = __builtin_elementwise_maximum(x, -200.0f);
  const float t = c * 1.44269504f;
  const float r = __builtin_fmaf(c, 1.92596303e-8f, __builtin_fmaf(c, 1.44269504f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e * 0.693147181f, r, e);
}

// s(l) and 1 - s(l).
__device__ __forceinline__ void sigmoid(float l, float& s, float& c) {
  const float t = exp_neg(-__builtin_fabsf(l));
  const float d = 1.0f / (1.0f + t), u = t * d;
  s = l < 0.0f ? u : d;
  c = l < 0.0f ? d : u;
}

// This lane's V logits from column c0 of a row; those past E are left alone.
template <bool BF16, int V>
__device__ __forceinline__ void load_logits(const void* row, int c0, int E, bool vec, float x[V]) {
  constexpr int N = 16 / (BF16 ? 2 : 4);           // elements of 16 bytes
  if (vec && c0 + V <= E) {
    if constexpr (BF16 && V == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + c0);
      x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
    } else {
#pragma unroll
      for (int i = 0; i < V / N; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const char*>(row) + (BF16 ? 2 : 4) * (c0 + N * i));
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (BF16) x[N * i + 2 * k] = bf16lo(q[k]), x[N * i + 2 * k + 1] = bf16hi(q[k]);
          else x[N * i + k] = __uint_as_float(q[k]);
        }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c0 + v < E)
        x[v] = BF16 ? bf16lo(static_cast<const uint16_t*>(row)[c0 + v]) : static_cast<const float*>(row)[c0 + v];
  }
}

// The row of this group of lanes: rows past the end take the last one (every lane
// stays active for the reductions) and store nothing.
template <int G>
__device__ __forceinline__ bool group_row(int64_t T, int64_t& row) {
  row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G;
  const bool live = row < T;
  if (!live) row = T - 1;
  return live;
}

template <bool BF16, int G, int V>
__global__ __launch_bounds__(256) void k_route(RouteArgs a) {
  static_assert(G >= 8 && G <= 64 && 256 % G == 0);
  const int lane = threadIdx.x & 63, g = lane & (G - 1);
  int64_t row;
  const bool live = group_row<G>(a.T, row);
  float x[V];
  load_logits<BF16, V>(static_cast<const char*>(a.logits) + row * a.ld * (BF16 ? 2 : 4), g * V, a.E, a.vec, x);
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = g * V + v < a.E ? order_key(x[v]) : 0u;
  int32_t* const ids = a.ids + row * a.top;
  float mine = 0.0f, first = 0.0f;                 // lane j: the j-th chosen logit
  for (int j = 0; j < a.top; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = m > key[v] ? m : key[v];
    const uint32_t best = group_max<G>(m);
    const uint64_t own = __ballot(m == best) >> (lane & ~(G - 1));
    if (g == __ffsll((unsigned long long)own) - 1) {
      int at = 0;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) at = key[v] == best ? v : at;
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = v == at ? 0u : key[v];
      if (live) ids[j] = g * V + at;
    }
    const float l = key_value(best);
    first = j == 0 ? l : first;
    mine = g == j ? l : mine;
  }
  const bool chosen = g < a.top;
  float w;
  if (a.sigmoid) {
    float s, c;
    sigmoid(mine, s, c);
    if (a.renorm) {
      const float top = __builtin_elementwise_minimum(first, 0.0f);
      const float e = exp_neg(__builtin_elementwise_minimum(mine, 0.0f) - top) / (1.0f + exp_neg(-__builtin_fabsf(mine)));
      w = e / group_sum<G>(chosen ? e : 0.0f);
      if (top == -INFINITY) w = 0.0f;
    } else {
      w = s;
    }
  } else {
    const float e = exp_neg(mine - first);
    float sum = chosen ? e : 0.0f;
    if (!a.renorm) {
      sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (g * V + v < a.E) sum = sum + exp_neg(x[v] - first);
    }
    w = e / group_sum<G>(sum);
    if (first == -INFINITY) w = 0.0f;
  }
  if (live && chosen) a.weights[row * a.top + g] = a.scale * w;
}

template <bool BF16, int G, int V>
__global__ __launch_bounds__(256) void k_route_backward(RouteArgs a) {
  const int lane = threadIdx.x & 63, g = lane & (G - 1), base = lane & ~(G - 1);
  int64_t row;
  const bool live = group_row<G>(a.T, row);
  const char* const logits = static_cast<const char*>(a.logits) + row * a.ld * (BF16 ? 2 : 4);
  const bool over_all = !a.sigmoid && !a.renorm;
  float x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = 0.0f;
  if (over_all) load_logits<BF16, V>(logits, g * V, a.E, a.vec, x);
  // lane j: the j-th choice (an id outside [0, E) takes no part)
  int id = -1;
  float dw = 0.0f, l = 0.0f;
  if (g < a.top) {
    id = a.ids[row * a.top + g];
    if ((uint32_t)id < (uint32_t)a.E) {
      dw = a.dweights[row * a.top + g];
      l = BF16 ? bf16lo(reinterpret_cast<const uint16_t*>(logits)[id]) : reinterpret_cast<const float*>(logits)[id];
    } else {
      id = -1;
    }
  }
  const bool chosen = id >= 0;
  float d = 0.0f, p[V];                            // d: the j-th choice's part of its logit's gradient
  float dot = 0.0f;
  if (a.sigmoid) {
    float s, c;
    sigmoid(l, s, c);
    if (a.renorm) {
      const float n = __builtin_elementwise_minimum(l, 0.0f);
      const float top = key_value(group_max<G>(chosen ? order_key(n) : order_key(-INFINITY)));
      const float e = exp_neg(n - top) / (1.0f + exp_neg(-__builtin_fabsf(l)));
      float q = e / group_sum<G>(chosen ? e : 0.0f);
      if (top == -INFINITY || !chosen) q = 0.0f;
      d = q * c * (dw - group_sum<G>(q * dw));
    } else {
      d = dw * (s * c);
    }
  } else if (!over_all) {
    const float top = key_value(group_max<G>(chosen ? order_key(l) : order_key(-INFINITY)));
    const float e = exp_neg(l - top);
    float q = e / group_sum<G>(chosen ? e : 0.0f);
    if (top == -INFINITY || !chosen) q = 0.0f;
    d = q * (dw - group_sum<G>(q * dw));
  } else {
    uint32_t m = 0u;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t k = g * V + v < a.E ? order_key(x[v]) : 0u;
      m = m > k ? m : k;
    }
    const float top = key_value(group_max<G>(m));
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = g * V + v < a.E ? exp_neg(x[v] - top) : 0.0f;
      sum = sum + p[v];
    }
    sum = group_sum<G>(sum);
    const float q = chosen ? exp_neg(l - top) / sum : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = top == -INFINITY ? 0.0f : p[v] / sum;
    dot = group_sum<G>(top == -INFINITY ? 0.0f : q * dw);
    d = dw;
  }
  float out[V];
#pragma unroll
  for (int v = 0; v < V; ++v) out[v] = 0.0f;
  for (int j = 0; j < a.top; ++j) {
    const int at = __shfl(chosen ? id : -1, base + j, 64) - g * V;
    const float dj = __shfl(d, base + j, 64);
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = at == v ? out[v] + dj : out[v];
  }
  if (!live) return;
  char* const dl = static_cast<char*>(a.dlogits) + row * a.ldd * (BF16 ? 2 : 4);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (g * V + v >= a.E) break;
    const float y = a.scale * (over_all ? p[v] * (out[v] - dot) : out[v]);
    if (BF16) reinterpret_cast<uint16_t*>(dl)[g * V + v] = (uint16_t)f32_to_bf16_rne(y);
    else reinterpret_cast<float*>(dl)[g * V + v] = y;
  }
}

template <bool BF16, int G, int V>
hipError_t launch_route_gv(const RouteArgs& a, hipStream_t st) {
  const unsigned wgs = (unsigned)((a.T * G + 255) / 256);
  RouteArgs b = a;
  const uintptr_t need = (BF16 && V == 4) ? 8 : 16;      // bytes of a lane's loads
  b.vec = (uintptr_t)a.logits % need == 0 && a.ld * (BF16 ? 2 : 4) % need == 0;
  if (a.dlogits) hipLaunchKernelGGL((k_route_backward<BF16, G, V>), dim3(wgs), dim3(256), 0, st, b);
  else hipLaunchKernelGGL((k_route<BF16, G, V>), dim3(wgs), dim3(256), 0, st, b);
  return hipGetLastError();
}

// The fewest lanes that hold the row at 4 logits each up to 64 experts and 8
// beyond (16 past 512), and at least one lane per choice.
template <bool BF16>
hipError_t launch_route_t(const RouteArgs& a, hipStream_t st) {
  const int t = a.top;
  if (a.E > 512) return launch_route_gv<BF16, 64, 16>(a, st);
  if (a.E > 64) {
    if (a.E > 256 || t > 32) return launch_route_gv<BF16, 64, 8>(a, st);
    if (a.E > 128 || t > 16) return launch_route_gv<BF16, 32, 8>(a, st);
    return launch_route_gv<BF16, 16, 8>(a, st);
  }
  if (t > 32) return launch_route_gv<BF16, 64, 4>(a, st);
  if (t > 16) return launch_route_gv<BF16, 32, 4>(a, st);
  if (a.E > 32 || t > 8) return launch_route_gv<BF16, 16, 4>(a, st);
  return launch_route_gv<BF16, 8, 4>(a, st);
}

// ---------------------------------------------------------------- sort by expert
constexpr int SORT_WAVES = 16, SORT_ROUNDS = 4;
constexpr int SORT_CHUNK = 64 * SORT_WAVES * SORT_ROUNDS;
constexpr int SORT_EMAX = 1024;
constexpr int64_t SORT_DIRECT = 64;

// Lanes whose slot has this lane's expert (live lanes only).
__device__ __forceinline__ uint64_t same_expert(int id, bool live, int bits) {
  uint64_t m = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const bool one = (id >> b) & 1;
    const uint64_t q = __ballot(one);
    m &= one ? q : ~q;
  }
  return m;
}

// LDS accesses of one wave keep this order (the hardware takes them in turn; this holds
// the compiler to it).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Slots of chunk blockIdx.x per expert: ws[chunk][E].
__global__ __launch_bounds__(64 * SORT_WAVES) void k_sort_count(SortArgs a) {
  __shared__ int cnt[SORT_EMAX];
  for (int e = threadIdx.x; e < a.E; e += 64 * SORT_WAVES) cnt[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 63;
  const int64_t s0 = (int64_t)blockIdx.x * SORT_CHUNK + (threadIdx.x >> 6) * (64 * SORT_ROUNDS) + lane;
  int id[SORT_ROUNDS];
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) id[r] = s0 + 64 * r < a.n ? a.ids[s0 + 64 * r] : -1;
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const bool live = (uint32_t)id[r] < (uint32_t)a.E;
    const uint64_t m = same_expert(id[r], live, a.bits);
    if (live && __ffsll((unsigned long long)m) - 1 == lane) atomicAdd(&cnt[id[r]], __popcll(m));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 64 * SORT_WAVES) a.ws[(int64_t)blockIdx.x * a.E + e] = cnt[e];
}

// ws[c][e] becomes the sum of chunks before c, ws[chunks][e] the total: one wave
// per expert.
__global__ __launch_bounds__(64) void k_sort_scan(SortArgs a) {
  const int lane = threadIdx.x, e = blockIdx.x;
  int carry = 0;
  for (int64_t c0 = 0; c0 < a.chunks; c0 += 64) {
    const int64_t c = c0 + lane;
    const int v = c < a.chunks ? a.ws[c * a.E + e] : 0;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(incl, d, 64);
      if (lane >= d) incl += u;
    }
    if (c < a.chunks) a.ws[c * a.E + e] = carry + incl - v;
    carry += __shfl(incl, 63, 64);
  }
  if (lane == 0) a.ws[a.chunks * a.E + e] = carry;
}

// Places the slots of chunk blockIdx.x; the counts of all chunks (their running
// sums if `scanned`) are in ws unless there is only one.
__global__ __launch_bounds__(64 * SORT_WAVES) void k_sort_place(SortArgs a, int scanned) {
  __shared__ uint16_t cnt[SORT_WAVES][SORT_EMAX];  // at most a chunk's 4096
  __shared__ int base[SORT_EMAX], tot[SORT_EMAX];
  __shared__ int end;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nt = blockDim.x;
  const int64_t chunk = blockIdx.x;
  const int64_t s0 = chunk * SORT_CHUNK + w * (64 * SORT_ROUNDS) + lane;
  int id[SORT_ROUNDS], at[SORT_ROUNDS];
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) id[r] = s0 + 64 * r < a.n ? a.ids[s0 + 64 * r] : -1;
  // the counts of all chunks, one per thread (the first of them requested here, beside
  // the ids): SORT_DIRECT * E of them at most
  const int counts = a.chunks > 1 && !scanned ? (int)a.chunks * a.E : 0;
  const int first = (int)threadIdx.x < counts ? a.ws[threadIdx.x] : 0;
  for (int e = lane; e < a.E; e += 64) cnt[w][e] = 0;
  for (int e = threadIdx.x; e < a.E; e += nt) base[e] = tot[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x, v = first; i < counts; v = (i += nt) < counts ? a.ws[i] : 0) {
    const int c = i / a.E, e = i - c * a.E;
    atomicAdd(&tot[e], v);                         // (whole numbers: any order gives the same sum)
    if (c < chunk) atomicAdd(&base[e], v);
  }
  // each slot's rank among its expert's in this wave, and the wave's counts
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const bool live = (uint32_t)id[r] < (uint32_t)a.E;
    const uint64_t m = same_expert(id[r], live, a.bits);
    const int before = __popcll(m & ((1ull << lane) - 1));
    const int seen = live ? cnt[w][id[r]] : 0;
    at[r] = seen + before;
    wave_fence();                                  // all lanes have read before the first one writes
    if (live && before == 0) cnt[w][id[r]] = (uint16_t)(seen + __popcll(m));
    wave_fence();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += nt) {
    int run = 0;
    for (int i = 0; i < nt / 64; ++i) {
      const int c = cnt[i][e];
      cnt[i][e] = (uint16_t)run;
      run += c;
    }
    if (scanned) {
      base[e] = a.ws[chunk * a.E + e];
      tot[e] = a.ws[a.chunks * a.E + e];
    } else if (counts == 0) {
      tot[e] = run;
    }
  }
  __syncthreads();
  if (w == 0) {                                    // group offsets: the exclusive sum of the totals
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane, v = e < a.E ? tot[e] : 0;
      int incl = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(incl, d, 64);
        if (lane >= d) incl += u;
      }
      if (e < a.E) {
        base[e] += carry + incl - v;
        if (chunk == 0) a.offsets[e] = carry + incl - v;
      }
      carry += __shfl(incl, 63, 64);
    }
    if (lane == 0) {
      end = carry;
      if (chunk == 0) a.offsets[a.E] = carry;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const int64_t s = s0 + 64 * r;
    if (s >= a.n) break;
    int d = -1;
    if ((uint32_t)id[r] < (uint32_t)a.E) {
      d = base[id[r]] + cnt[w][id[r]] + at[r];
      a.rows[d] = (int32_t)((uint32_t)s / (uint32_t)a.top);
    }
    a.dest[s] = d;
    if (s >= end) a.rows[s] = -1;                  // past the last sorted row
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
  return a.bf16 ? launch_route_t<true>(a, st) : launch_route_t<false>(a, st);
}

size_t sort_workspace(int64_t n, int32_t E) {
  const int64_t chunks = (n + SORT_CHUNK - 1) / SORT_CHUNK;
  return chunks > 1 ? (size_t)(chunks + 1) * E * sizeof(int) : 0;
}

hipError_t launch_expert_sort(const SortArgs& args, hipStream_t st) {
  SortArgs a = args;
  a.chunks = (a.n + SORT_CHUNK - 1) / SORT_CHUNK;
  if (a.chunks < 1) a.chunks = 1;                  // no slots: the offsets are still written
  a.bits = 0;
  while ((1 << a.bits) < a.E) ++a.bits;
  const int64_t waves = a.chunks > 1 ? SORT_WAVES : (a.n + 64 * SORT_ROUNDS - 1) / (64 * SORT_ROUNDS);
  const unsigned nt = 64 * (unsigned)(waves < 1 ? 1 : waves);
  const bool scan = a.chunks > SORT_DIRECT;
  if (a.chunks > 1)
    hipLaunchKernelGGL(k_sort_count, dim3((unsigned)a.chunks), dim3(64 * SORT_WAVES), 0, st, a);
  if (scan) hipLaunchKernelGGL(k_sort_scan, dim3((unsigned)a.E), dim3(64), 0, st, a);
  hipLaunchKernelGGL(k_sort_place, dim3((unsigned)a.chunks), dim3(nt), 0, st, a, (int)scan);
  return hipGetLastError();
}

}  // namespace mx
