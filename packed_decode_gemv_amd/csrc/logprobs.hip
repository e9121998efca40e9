// Log probabilities of given tokens, entropies and the most likely tokens of rows of
// logits, in one pass over them (meaning in vbq.h).
//
// A wavefront takes steps of 2048 logits, 32 a lane, and keeps m (its maximum), s =
// sum of e and t = sum of e (x - m) with e = exp(x - m), from which lse = m + log s and
// the entropy = log s - t / s. For the most likely tokens it keeps a list in LDS of
// 64-bit keys (the value's order, then the lowest index), and T, the top-th largest
// key of those met: a step with nothing above T costs one comparison a lane, others
// append what is above, and the list is cut back to `top` when it passes 64. Keys
// never tie, so what is kept does not depend on the order in which it is met.
//   In the first step T is the top-th largest of the lanes' own best (that many keys
// are no smaller), so few are appended.
//   The wavefronts of a workgroup are joined in LDS, the workgroups of a row by the
// last of them that finishes.
#include "logprobs.h"

namespace vbq {
namespace {

constexpr int kWaves = kLogprobSteps;
constexpr int kPer = kLogprobStep / 64;       // logits of a lane and step
constexpr int kGroup8 = kPer / 8;
constexpr int kTop = VBQ_LOGPROBS_MAX_TOP;
constexpr int kKeep = 64;                     // a list longer than this is cut back
constexpr int kList = kKeep + 8 * 64;         // places: what 64 lanes append of eight values each
constexpr float kLog2e = 1.44269504088896341f;

// Order of a float as an unsigned number (zeros of both signs are one number), then
// the lowest index.
__device__ inline uint64_t key_of(float x, uint32_t index) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x == 0.f ? 0.f : x);
  const uint32_t o = u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return (uint64_t)o << 32 | (0xFFFFFFFFu - index);
}
__device__ inline float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ inline uint32_t key_index(uint64_t k) { return 0xFFFFFFFFu - (uint32_t)k; }

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ inline uint64_t lane_key(uint64_t v, int i) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, i);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), i);
  return (uint64_t)hi << 32 | lo;
}
// What a wavefront wrote to LDS is read by its other lanes afterwards.
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Keys of a lane that are larger than its own, over the 64 lanes.
__device__ inline int lanes_above(uint64_t key) {
  int n = 0;
#pragma unroll 16
  for (int i = 0; i < 64; ++i) n += lane_key(key, i) > key;
  return n;
}

// The n keys of `list`, cut back to the `top` largest, largest first.
__device__ inline int cut(uint64_t* list, int n, int top, uint32_t lane) {
  wave_sync();
  constexpr int MINE = (kList + 63) / 64;
  uint64_t key[MINE];
  int above[MINE];
#pragma unroll
  for (int j = 0; j < MINE; ++j) {
    key[j] = 64 * j + (int)lane < n ? list[64 * j + lane] : 0;
    above[j] = 0;
  }
  if (n <= 64) {
    for (int i = 0; i < n; ++i) above[0] += lane_key(key[0], i) > key[0];
  } else {
    for (int i = 0; i < n; ++i) {
      const uint64_t o = list[i];
#pragma unroll
      for (int j = 0; j < MINE; ++j) above[j] += o > key[j];
    }
  }
  wave_sync();
#pragma unroll
  for (int j = 0; j < MINE; ++j)
    if (64 * j + (int)lane < n && above[j] < top) list[above[j]] = key[j];
  wave_sync();
  return min(n, top);
}

// Two parts of a row as one.
__device__ inline void join(LogprobPart& a, const LogprobPart& b) {
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf(a.m - m, -1000.f), db = fmaxf(b.m - m, -1000.f);
  const float fa = __builtin_amdgcn_exp2f(da * kLog2e), fb = __builtin_amdgcn_exp2f(db * kLog2e);
  a.t = fa * __builtin_fmaf(da, a.s, a.t) + fb * __builtin_fmaf(db, b.s, b.t);
  a.s = fa * a.s + fb * b.s;
  a.m = m;
  a.before += b.before;
}

// One wavefront's way through its part of a row.
struct Walk {
  float m, s, t;           // m: the wavefront's; s, t: the lane's
  uint64_t least;          // T: keys up to it are not wanted
  float least_value;
  int n;                   // keys in the list
  int before;              // (a lane's count)
  uint64_t* list;
  int top;
  uint32_t lane;
  float given;             // the given token's logit
  uint32_t token;

  // N values of a lane, value i at index(i), of which the first step may hold too few
  // lanes (valid(i) is false: the value is minus infinity and its key 0).
  template <int N, class Index, class Valid>
  __device__ inline void step(const float (&x)[N], Index index, Valid valid, bool count, uint32_t lowest,
                              uint32_t highest) {
    constexpr int GROUPS = (N + 7) / 8;
    float best[GROUPS], top_x = -__builtin_inff();
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      best[g] = x[8 * g];
#pragma unroll
      for (int i = 8 * g + 1; i < N && i < 8 * g + 8; ++i) best[g] = fmaxf(best[g], x[i]);
      top_x = fmaxf(top_x, best[g]);
    }
    if (__any(top_x > m)) {   // sums follow the maximum
      const float to = wave_max(fmaxf(top_x, m)), d = fmaxf(m - to, -1000.f), f = __builtin_amdgcn_exp2f(d * kLog2e);
      t = f * __builtin_fmaf(d, s, t);
      s *= f;
      m = to;
    }
    if (top && (n < top || __any(top_x > least_value))) {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const uint64_t over = __ballot(best[g] > least_value);
        if (n >= top && !over) continue;
        uint64_t key[8], mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          key[i] = 8 * g + i < N && valid(8 * g + i) ? key_of(x[8 * g + i < N ? 8 * g + i : 0], index(8 * g + i)) : 0;
          mine = key[i] > mine ? key[i] : mine;
        }
        uint64_t above = least;   // what is wanted is larger
        if (__builtin_popcountll(__ballot(mine > least)) > top) {
          const uint64_t place = __ballot(lanes_above(mine) == top - 1);
          if (place) {   // (not where many lanes hold nothing)
            const uint64_t at = lane_key(mine, __builtin_ctzll(place));
            above = at > above ? at - 1 : above;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool want = key[i] > above;
          const uint64_t who = __ballot(want);
          if (!who) continue;
          if (want) list[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0))] = key[i];
          n += __builtin_popcountll(who);
        }
        if (n > kKeep || (!least && n >= top)) {
          n = cut(list, n, top, lane);
          least = list[top - 1];
          least = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(least >> 32)) << 32 |
                  (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)least);
          least_value = key_value(least);
        }
      }
    }
    if (count) {
      if (highest < token) {
#pragma unroll
        for (int i = 0; i < N; ++i) before += x[i] >= given && valid(i);
      } else if (lowest > token) {
#pragma unroll
        for (int i = 0; i < N; ++i) before += x[i] > given;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) before += x[i] > given || (x[i] == given && index(i) < token && valid(i));
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = x[i] - m, e = __builtin_amdgcn_exp2f(d * kLog2e);
      s += e;
      t = __builtin_fmaf(e, fmaxf(d, -1000.f), t);   // (0 where e is 0, and d perhaps infinite)
    }
  }
};

template <int DT>
__device__ inline float value_at(const void* row, int64_t i) {
  if constexpr (DT == VBQ_F32) return static_cast<const float*>(row)[i];
  const uint16_t u = static_cast<const uint16_t*>(row)[i];
  if constexpr (DT == VBQ_F16) return (float)__builtin_bit_cast(_Float16, u);
  return __builtin_bit_cast(float, (uint32_t)u << 16);
}

template <int DT>
__global__ __launch_bounds__(64 * kWaves) void k_token_logprobs(Logprobs a) {
  constexpr int PER16 = DT == VBQ_F32 ? 4 : 8, VECS = kPer / PER16;   // logits of a load, loads of a step
  __shared__ uint64_t lists[kWaves][kList];
  __shared__ LogprobPart wave_part[kWaves];
  __shared__ int counts[kWaves];
  __shared__ uint32_t last;
  const uint32_t tid = threadIdx.x, lane = tid & 63u;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = blockIdx.x / (uint32_t)a.splits;
  const int split = (int)(blockIdx.x % (uint32_t)a.splits);
  const void* const x = DT == VBQ_F32 ? (const void*)(static_cast<const float*>(a.logits) + row * a.row_stride)
                                      : (const void*)(static_cast<const uint16_t*>(a.logits) + row * a.row_stride);
  // The row's first logits up to a multiple of 16 bytes, its loads of 16 bytes, the rest.
  constexpr int SIZE = DT == VBQ_F32 ? 4 : 2;
  const int head = min(a.vocab, (int)((16u - ((uint32_t)reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / SIZE);
  const int vecs = (a.vocab - head) / PER16, tail = a.vocab - head - vecs * PER16;
  const u32x4* const body = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(x) + head * SIZE);

  Walk w;
  w.m = -__FLT_MAX__;
  w.s = w.t = 0.f;
  w.least = 0;
  w.least_value = -__builtin_inff();
  w.n = w.before = 0;
  w.list = lists[wave];
  w.top = a.top;
  w.lane = lane;
  w.given = 0.f;
  int64_t token = -1;
  if (a.tokens) token = a.long_tokens ? static_cast<const int64_t*>(a.tokens)[row] : static_cast<const int32_t*>(a.tokens)[row];
  const bool count = token >= 0 && token < a.vocab;
  w.token = count ? (uint32_t)token : 0u;
  if (count) w.given = value_at<DT>(x, token);

  const bool edges = split == 0 && wave == 0;
  auto edge = [&](int first, int many) {   // fewer than eight logits, one a lane
    float v[1] = {-__builtin_inff()};
    if ((int)lane < many) v[0] = value_at<DT>(x, first + (int)lane);
    w.step(v, [&](int) { return (uint32_t)first + lane; }, [&](int i) { return i == 0 && (int)lane < many; }, count,
           (uint32_t)first, (uint32_t)(first + many - 1));
  };
  if (edges && head) edge(0, head);
  const int steps = (vecs + 64 * VECS - 1) / (64 * VECS);
  for (int j = split * kWaves + wave; j < steps; j += a.splits * kWaves) {
    const int v0 = j * (64 * VECS);
    u32x4 raw[VECS];
    float v[kPer];
    const bool whole = v0 + 64 * VECS <= vecs;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      raw[i] = u32x4{0, 0, 0, 0};
      if (whole || v0 + 64 * i + (int)lane < vecs) raw[i] = body[v0 + 64 * i + lane];
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t u = raw[i][c];
        if constexpr (DT == VBQ_F32) {
          v[PER16 * i + c] = __builtin_bit_cast(float, u);
        } else if constexpr (DT == VBQ_F16) {
          const half2_t h = __builtin_bit_cast(half2_t, u);
          v[PER16 * i + 2 * c] = (float)h.x;
          v[PER16 * i + 2 * c + 1] = (float)h.y;
        } else {
          v[PER16 * i + 2 * c] = __builtin_bit_cast(float, u << 16);
          v[PER16 * i + 2 * c + 1] = __builtin_bit_cast(float, u & 0xFFFF0000u);
        }
      }
    }
    if (!whole) {
#pragma unroll
      for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int c = 0; c < PER16; ++c)
          v[PER16 * i + c] = v0 + 64 * i + (int)lane < vecs ? v[PER16 * i + c] : -__builtin_inff();
    }
    const uint32_t first = (uint32_t)(head + v0 * PER16);
    w.step(v, [&](int i) { return first + (uint32_t)((64 * (i / PER16) + (int)lane) * PER16 + i % PER16); },
           [&](int i) { return whole || v0 + 64 * (i / PER16) + (int)lane < vecs; }, count, first,
           first + (uint32_t)(min(64 * VECS, vecs - v0) * PER16 - 1));
  }
  if (edges && tail) edge(a.vocab - tail, tail);

  // The workgroup's part: sums, and the largest keys of the wavefronts' lists.
  if (a.top) w.n = cut(w.list, w.n, a.top, lane);
  LogprobPart part = {w.m, wave_sum(w.s), wave_sum(w.t), (int)wave_total((uint32_t)w.before)};
  if (lane == 0) {
    wave_part[wave] = part;
    counts[wave] = w.n;
  }
  __syncthreads();
  part = wave_part[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) join(part, wave_part[i]);
  // keys of this thread: up to kTop of each wavefront
  static_assert(kWaves * kTop <= 64 * kWaves, "a thread a key");
  uint64_t key = 0;
  int above = 0;
  if ((int)tid < kWaves * a.top) {
    const int from = (int)tid / a.top, at = (int)tid % a.top;
    if (at < counts[from]) {
      key = lists[from][at];
      for (int i = 0; i < kWaves; ++i)
        for (int c = 0; c < counts[i]; ++c) above += lists[i][c] > key;
    }
  }

  const bool wants = key && above < a.top;
  if (a.splits > 1) {
    // (device-scope stores, waited for before the count; read by device-scope loads)
    uint64_t* const keys = a.keys + (row * a.splits + split) * a.top;
    if (wants) __hip_atomic_store(keys + above, key, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    int held = 0;
    for (int i = 0; i < kWaves; ++i) held += counts[i];
    if ((int)tid >= held && (int)tid < a.top) __hip_atomic_store(keys + tid, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (tid == 0) {
      uint64_t* const p = reinterpret_cast<uint64_t*>(a.parts + row * a.splits + split);
      const u32x4 raw = __builtin_bit_cast(u32x4, part);
      __hip_atomic_store(p, (uint64_t)raw.y << 32 | raw.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(p + 1, (uint64_t)raw.w << 32 | raw.z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __builtin_amdgcn_s_waitcnt(VBQ_VMCNT_IMM(0));
    __syncthreads();
    if (tid == 0) {
      last = __hip_atomic_fetch_add(a.counters + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(a.splits - 1);
      if (last) __hip_atomic_store(a.counters + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!last) return;
    // Each wavefront takes the keys of every fourth part, then the four are joined as above.
    if (a.top) {
      int n = 0;
      const uint64_t* const from = a.keys + row * a.splits * a.top;
      for (int p = wave; p < a.splits; p += kWaves) {
        uint64_t k = 0;
        if ((int)lane < a.top) k = __hip_atomic_load(from + p * a.top + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint64_t who = __ballot(k != 0);   // (a part of few logits has fewer keys)
        if (k) w.list[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0))] = k;
        n += __builtin_popcountll(who);
      }
      static_assert((kLogprobSplits + kWaves - 1) / kWaves * kTop <= kList, "the parts' keys fit a list");
      n = cut(w.list, n, a.top, lane);
      if (lane == 0) counts[wave] = n;
    }
    if (wave == 0) {   // sums: a part a lane
      LogprobPart q = {-__FLT_MAX__, 0.f, 0.f, 0};
      if ((int)lane < a.splits) {
        const uint64_t* const p = reinterpret_cast<const uint64_t*>(a.parts + row * a.splits + lane);
        const uint64_t u = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint64_t v = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        q = __builtin_bit_cast(LogprobPart, (u32x4{(uint32_t)u, (uint32_t)(u >> 32), (uint32_t)v, (uint32_t)(v >> 32)}));
      }
      const float m = wave_max(q.m), d = fmaxf(q.m - m, -1000.f), f = __builtin_amdgcn_exp2f(d * kLog2e);
      part = {m, wave_sum(f * q.s), wave_sum(f * __builtin_fmaf(d, q.s, q.t)), (int)wave_total((uint32_t)q.before)};
      if (lane == 0) wave_part[0] = part;
    }
    __syncthreads();
    part = wave_part[0];
    key = 0;
    above = 0;
    if ((int)tid < kWaves * a.top) {
      const int from = (int)tid / a.top, at = (int)tid % a.top;
      if (at < counts[from]) {
        key = lists[from][at];
        for (int i = 0; i < kWaves; ++i)
          for (int c = 0; c < counts[i]; ++c) above += lists[i][c] > key;
      }
    }
  }

  // Answers. A sum that is no number: the row holds a NaN or an infinity above all.
  const bool bad = part.s != part.s;
  const float log_s = logf(part.s);
  if (tid == 0) {
    const float nan = __builtin_nanf("");
    if (a.lse) a.lse[row] = bad ? nan : part.s == 0.f ? -__builtin_inff() : part.m + log_s;
    if (a.entropy) a.entropy[row] = bad ? nan : part.s == 0.f ? 0.f : log_s - part.t / part.s;
    if (a.tokens) {
      const bool there = count && !bad;
      a.logprob[row] = !there ? nan : part.s == 0.f ? -__builtin_inff() : (w.given - part.m) - log_s;
      a.rank[row] = there ? part.before : -1;
    }
  }
  if ((int)tid < a.top && bad) {
    a.top_logprob[row * a.top + tid] = __builtin_nanf("");
    a.top_index[row * a.top + tid] = -1;
  }
  if (key && above < a.top && !bad) {
    const float v = key_value(key);
    a.top_logprob[row * a.top + above] = part.s == 0.f ? -__builtin_inff() : (v - part.m) - log_s;
    a.top_index[row * a.top + above] = (int32_t)key_index(key);
  }
}

}  // namespace

int logprob_splits(int rows, int vocab) {
  const int64_t steps = ((int64_t)vocab + kLogprobStep - 1) / kLogprobStep, most = (steps + kWaves - 1) / kWaves;
  int64_t n = 2 * VBQ_LOGPROBS_COUNTERS / rows;   // (more than one for as many rows as there are counters at most)
  n = n < most ? n : most;
  return (int)(n < 1 ? 1 : n < kLogprobSplits ? n : kLogprobSplits);
}

hipError_t launch_token_logprobs(const Logprobs& a, int dtype, hipStream_t s) {
  const int64_t groups = (int64_t)a.rows * a.splits;
  if (groups == 0) return hipSuccess;
  if (groups * (64 * kWaves) > (int64_t)UINT32_MAX) return hipErrorNotSupported;
  const dim3 grid((uint32_t)groups);
  if (dtype == VBQ_F16) k_token_logprobs<VBQ_F16><<<grid, 64 * kWaves, 0, s>>>(a);
  else if (dtype == VBQ_BF16) k_token_logprobs<VBQ_BF16><<<grid, 64 * kWaves, 0, s>>>(a);
  else k_token_logprobs<VBQ_F32><<<grid, 64 * kWaves, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace vbq
