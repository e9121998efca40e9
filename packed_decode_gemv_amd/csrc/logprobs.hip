// Log probabilities of given tokens, entropies and the most likely tokens of rows of
// logits, in one pass over them (meaning in vbq.h).
//
// A wavefront takes steps of 1024 logits, 16 a lane, the next one's on their way while
// one is worked on. In base two, with b = m log2(e) for the wavefront's maximum m, it
// keeps s = sum of e and t = sum of e y with e = 2^y, y = x log2(e) - b (one fma: the
// rounding of b is the same for all, and leaves the logarithms again), from which
// lse = m + ln2 log2 s (here it stays, 2^-24 m at most), logprob = ln2 (y - log2 s) and
// entropy = ln2 (log2 s - t / s).
//   For the most likely tokens it keeps a list in LDS of 64-bit keys (the value's
// order, then the lowest index), and `least`, the top-th largest key of those met.
// Indexes rise from step to step, so a value is wanted only if it is larger than
// least's was before the step: a step with none costs one comparison a lane. Others
// append what is above least, and the list is cut back to `top` when it passes 64.
// Keys never tie, so what is kept does not depend on the order in which it is met. In
// the first step the top-th largest of the lanes' own best is a bound that few pass.
//   The wavefronts of a workgroup are joined in LDS, the workgroups of a row by the
// last of them that finishes.
//   Many fp32 rows are bound by memory: 2047 of 128256 (1.05 GB), top 5, take 185 us,
// 5.7 TB/s, with vector instructions 60 to 70% of that time beside it; in 16 bits they bind, 91%
// busy: 117 us (4.5 TB/s; 104 without a list). What did not help the first: a row's first and
// last logits loaded in the step that takes them 189; then a bound shared by a row's wavefronts
// 188, but 64 rows of 32001 18.7 and 19.2 for 17.7; registers for six and eight wavefronts a SIMD
// 206 and 205. Few rows are a chain of one step and two joins: one row of 128256, top 20,
// 13.3 us, of which the first step 3.5, the joins 2 each.
#include "logprobs.h"

namespace vbq {
namespace {

constexpr int kWaves = 4;                     // of a workgroup
constexpr int kPer = kLogprobStep / 64;       // logits of a lane and step
constexpr int kTop = VBQ_LOGPROBS_MAX_TOP;
constexpr int kKeep = 64, kSpare = 16;        // a list is cut back when it passes `top` by so many, or 64
constexpr int kList = kKeep + 64;             // places: a wavefront appends 64 keys at a time
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// Order of a float as an unsigned number (zeros of both signs are one number), then
// the lowest index.
__device__ inline uint32_t order_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x == 0.f ? 0.f : x);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t kZero = 0x80000000u, kMinusInfinity = 0x007FFFFFu;   // in that order
__device__ inline float value_of(uint32_t order) {
  return __builtin_bit_cast(float, order ^ ((order >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ inline float just_below(uint32_t order) { return value_of(order - (order == kZero ? 2u : 1u)); }
__device__ inline uint64_t key_of(float x, uint32_t index) {
  return (uint64_t)order_of(x) << 32 | (0xFFFFFFFFu - index);
}
__device__ inline float key_value(uint64_t k) { return value_of((uint32_t)(k >> 32)); }
__device__ inline uint32_t key_index(uint64_t k) { return 0xFFFFFFFFu - (uint32_t)k; }

// A maximum in base two, b. What rounding leaves of m log2(e) is in every exponent of its
// sums: up to 2^30 64 at most, so that sums of 2^30 terms, and these times it, stay within
// 2^101. From 2^30 on (far) b is m itself: there numbers that are not equal are 64 apart at
// least, further than 2^y or exp reach beside 1 (2^30 terms of 2^-64).
__device__ inline bool is_far(float m) { return !(fabsf(m) < 0x1p30f); }
__device__ inline float to_base(float m) { return is_far(m) ? m : m * kLog2e; }
// log2 of what sums on one maximum are worth on another, as large or larger: not below
// -1000, so that nothing times its power is no number. Of two kinds they are 64 apart too.
__device__ inline float down(float from, float to) {
  const float d = is_far(from) == is_far(to) ? to_base(from) - to_base(to) : -1000.f;
  return fmaxf(d, -1000.f);
}

// Over the wavefront, the result in every lane: within rows of 16 lanes, then rows.
template <class Op>
__device__ inline uint32_t wave_reduce(uint32_t v, uint32_t neutral, Op op) {
#define VBQ_STEP(CTRL, ROWS) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)neutral, (int)v, CTRL, ROWS, 0xF, false))
  VBQ_STEP(0x111, 0xF);   // row_shr:1, 2, 4, 8
  VBQ_STEP(0x112, 0xF);
  VBQ_STEP(0x114, 0xF);
  VBQ_STEP(0x118, 0xF);
  VBQ_STEP(0x142, 0xA);   // row_bcast:15 into rows 1 and 3
  VBQ_STEP(0x143, 0xC);   // row_bcast:31 into rows 2 and 3
#undef VBQ_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ inline uint32_t as_bits(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ inline float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ inline float wave_max(float v) {
  return as_float(wave_reduce(as_bits(v), as_bits(-__builtin_inff()),
                              [](uint32_t x, uint32_t y) { return as_bits(fmaxf(as_float(x), as_float(y))); }));
}
__device__ inline float wave_sum(float v) {
  return as_float(wave_reduce(as_bits(v), 0u, [](uint32_t x, uint32_t y) { return as_bits(as_float(x) + as_float(y)); }));
}
__device__ inline uint32_t wave_min(uint32_t v) {
  return wave_reduce(v, 0xFFFFFFFFu, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
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

// The most likely tokens that a wavefront has met.
struct Best {
  uint64_t* list;
  uint64_t least;   // keys up to it are not wanted
  int n, top, limit;   // cut back when there are more than `limit`
  uint32_t lane;
  int sorted;       // keys in order at the list's head

  // Cuts the list back to the `top` largest keys, largest first.
  __device__ inline void cut() {
    if (n == sorted) return;
    wave_sync();
    const uint64_t a = (int)lane < n ? list[lane] : 0;
    int above = 0;   // (lanes beyond n hold 0, larger than nothing)
    if (n <= 64) {
      for (int i = 0; i < n; i += 8)
#pragma unroll
        for (int c = 0; c < 8; ++c) above += lane_key(a, i + c) > a;
      if (above < top && a) list[above] = a;
      wave_sync();
      if (n >= top) least = lane_key(a, __builtin_ctzll(__ballot(a && above == top - 1)));
    } else {
      const uint64_t b = 64 + (int)lane < n ? list[64 + lane] : 0;
      int above_b = 0;
      for (int i = 0; i < 64; i += 4)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint64_t o = lane_key(a, i + c), q = lane_key(b, i + c);
          above += (o > a) + (q > a);
          above_b += (o > b) + (q > b);
        }
      wave_sync();
      if (above < top) list[above] = a;
      if (above_b < top && b) list[above_b] = b;
      wave_sync();
      least = list[top - 1];
      least = lane_key(least, 0);
    }
    n = min(n, top);
    sorted = n;
  }
  // Keys of a lane (0: none) that are wanted.
  __device__ inline void offer(uint64_t key) {
    const bool want = key > least;
    const uint64_t who = __ballot(want);
    if (!who) return;
    if (want) list[n + lanes_below(who)] = key;
    n += __builtin_popcountll(who);
    if (n > limit) cut();
  }
};

// Two parts of a row as one.
__device__ inline void join(LogprobPart& a, const LogprobPart& b) {
  const float m = fmaxf(a.m, b.m), da = down(a.m, m), db = down(b.m, m);
  const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
  a.t = fa * __builtin_fmaf(da, a.s, a.t) + fb * __builtin_fmaf(db, b.s, b.t);
  a.s = fa * a.s + fb * b.s;
  a.m = m;
  a.before += b.before;
}

// One wavefront's way through its part of a row.
struct Walk {
  float m, s, t;           // m: the wavefront's; s, t: the lane's
  float mul, add;          // y = mul x + add
  Best best;
  bool count;              // a token is given: its logit and number
  float given;
  uint32_t token;
  int before;              // logits before it

  // N values of a lane, value i at index(i); where valid(i) is false it is minus
  // infinity and stands for nothing (full: nowhere). The step's indexes are lowest ..
  // highest (full), or any (edge: lower ones than have been met too).
  template <int PER16, int N, class Index, class Valid>
  __device__ inline void step(const float (&x)[N], Index index, Valid valid, bool full, bool edge,
                              uint32_t lowest, uint32_t highest) {
    float high = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) high = fmaxf(high, x[i]);
    if (__any(high > m)) {   // sums follow the maximum
      const float to = wave_max(fmaxf(high, m)), d = down(m, to), f = __builtin_amdgcn_exp2f(d);
      t = f * __builtin_fmaf(d, s, t);
      s *= f;
      m = to;
      mul = is_far(m) ? 1.f : kLog2e;
      add = -to_base(m);
    }
    if (best.top) {
      // (until the list has been full: a bound that `top` of the lanes' best reach at
      // least, to 1/512 of their range)
      const bool open = best.least == 0;
      float bound = key_value(best.least);
      bool all = false;
      if (open) {
        const uint32_t o = order_of(high);
        const bool finite = o > kMinusInfinity;
        all = __builtin_popcountll(__ballot(finite)) < best.top;
        if (!all) {
          uint32_t low = wave_min(finite ? o : 0xFFFFFFFFu);
          const uint32_t range = ~wave_min(~o) - low;
          uint32_t bit = range ? 0x80000000u >> __builtin_clz(range) : 0u;
          for (int i = 0; i < 9 && bit; ++i, bit >>= 1)
            if (__builtin_popcountll(__ballot(o >= low + bit)) >= best.top) low += bit;
          bound = just_below(low);
        } else {
          bound = -__builtin_inff();
        }
      } else if (edge) {   // (as large is enough, for a lower index)
        const uint32_t low = order_of(bound);
        all = low <= kMinusInfinity;
        bound = all ? -__builtin_inff() : just_below(low);
      }
      if (open || all || __any(high > bound)) {
        uint32_t hits = 0;   // of the lane's values; one of each lane is taken at a time
#pragma unroll
        for (int i = 0; i < N; ++i) hits |= (x[i] > bound ? 1u : 0u) << i;
        // (of equal numbers the lowest indexes will do: those of the first eight lanes' first load)
        if (all && (edge || best.lane < 8)) hits |= (1u << (edge ? 1 : PER16)) - 1u;
        while (__any(hits != 0)) {
          const int i = hits ? __builtin_ctz(hits) : 0;
          float part[N];
#pragma unroll
          for (int c = 0; c < N; ++c) part[c] = x[c];
#pragma unroll
          for (int d = 1; d < N; d <<= 1)
#pragma unroll
            for (int c = 0; c < N; c += 2 * d) part[c] = i & d ? part[c + d] : part[c];
          const float v = part[0];
          best.offer(hits && valid(i) ? key_of(v, index(i)) : 0);
          hits &= hits - 1;
        }
        if (open) best.cut();
      }
    }
    if (count) {
      if (!edge && (lowest > token || (highest < token && full))) {
        const float least = lowest > token ? value_of(order_of(given) + 1) : given;   // larger, or as large
#pragma unroll
        for (int i = 0; i < N; ++i) before += __builtin_popcountll(__ballot(x[i] >= least));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          before += __builtin_popcountll(__ballot(x[i] > given || (x[i] == given && index(i) < token && valid(i))));
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y = __builtin_fmaf(x[i], mul, add), e = __builtin_amdgcn_exp2f(y);
      s += e;
      t = __builtin_fmaf(e, fmaxf(y, -1000.f), t);   // (0 where e is 0, and y perhaps infinite)
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

// ROW_WAVES: wavefronts that share a row (or a part of one): all of a workgroup, or one.
template <int DT, int ROW_WAVES>
__global__ __launch_bounds__(64 * kWaves) void k_token_logprobs(Logprobs a) {
  constexpr int PER16 = DT == VBQ_F32 ? 4 : 8, VECS = kPer / PER16;   // logits of a load, loads of a step
  constexpr int SIZE = DT == VBQ_F32 ? 4 : 2;
  __shared__ uint64_t lists[kWaves][kList];
  __shared__ LogprobPart wave_part[kWaves];
  __shared__ int counts[kWaves];
  __shared__ uint32_t last;
  const uint32_t tid = threadIdx.x, lane = tid & 63u;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = ROW_WAVES == 1 ? (int64_t)blockIdx.x * kWaves + wave : (int64_t)(blockIdx.x / (uint32_t)a.splits);
  if (ROW_WAVES == 1 && row >= a.rows) return;
  const int split = ROW_WAVES == 1 ? 0 : (int)(blockIdx.x % (uint32_t)a.splits);
  const uint8_t* const x = static_cast<const uint8_t*>(a.logits) + row * a.row_stride * SIZE;
  int64_t token = -1;
  if (a.tokens) token = a.long_tokens ? static_cast<const int64_t*>(a.tokens)[row] : static_cast<const int32_t*>(a.tokens)[row];
  // The row's first logits up to a multiple of 16 bytes, its loads of 16 bytes, the rest.
  const int head = min(a.vocab, (int)((16u - ((uint32_t)reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / SIZE);
  const int vecs = (a.vocab - head) / PER16, tail = a.vocab - head - vecs * PER16;
  const u32x4* const body = reinterpret_cast<const u32x4*>(x + head * SIZE);
  const int steps = (vecs + 64 * VECS - 1) / (64 * VECS), stride = a.splits * ROW_WAVES;
  u32x4 raw[VECS];
  auto load = [&](int j) {
    const u32x4* const at = body + (int64_t)j * (64 * VECS) + lane;
    const int left = vecs - j * (64 * VECS) - (int)lane;
    if ((j + 1) * (64 * VECS) <= vecs) {
#pragma unroll
      for (int i = 0; i < VECS; ++i) raw[i] = at[64 * i];
    } else {
#pragma unroll
      for (int i = 0; i < VECS; ++i) raw[i] = 64 * i < left ? at[64 * i] : u32x4{0, 0, 0, 0};
    }
  };
  int j = split * ROW_WAVES + (ROW_WAVES == 1 ? 0 : wave);
  if (j < steps) load(j);

  Walk w;
  w.m = -__FLT_MAX__;
  w.mul = 1.f;
  w.add = -w.m;
  w.s = w.t = 0.f;
  w.before = 0;
  w.best = Best{lists[wave], 0, 0, a.top, min(a.top + kSpare, kKeep), lane, 0};
  w.count = token >= 0 && token < a.vocab;
  w.token = w.count ? (uint32_t)token : 0u;
  w.given = w.count ? value_at<DT>(x, token) : 0.f;

  // Steps of this wavefront, those of whole loads first; the row's first and last logits,
  // one a lane, are the step after the last of them.
  bool edges = (head || tail) && steps % stride == split * ROW_WAVES + (ROW_WAVES == 1 ? 0 : wave);
  float edge_value = -__builtin_inff();
  const uint32_t edge_at = (int)lane < head ? lane : (uint32_t)(a.vocab - (head + tail)) + lane;
  if (edges && (int)lane < head + tail) edge_value = value_at<DT>(x, edge_at);
  while (j < steps || edges) {
    float v[kPer];
    uint32_t at, first;        // the lane's first logit, the step's
    int left, values = kPer;   // loads, and values of a lane
    bool whole = false;
    const bool edge = j >= steps;
    if (edge) {
      left = head + tail;
      first = 0;
      at = edge_at;
      values = 1;
#pragma unroll
      for (int i = 1; i < kPer; ++i) v[i] = -__builtin_inff();
      v[0] = edge_value;
      edges = false;
    } else {
      const int v0 = j * (64 * VECS);
      left = vecs - v0;
      whole = left >= 64 * VECS;
      first = (uint32_t)(head + v0 * PER16);
      at = first + lane * PER16;
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
            v[PER16 * i + c] = 64 * i + (int)lane < left ? v[PER16 * i + c] : -__builtin_inff();
      }
      j += stride;
      if (j < steps) load(j);
    }
    w.step<PER16>(v, [&](int i) { return at + (uint32_t)(64 * PER16 * (i / PER16) + i % PER16); },
           [&](int i) { return whole || (i < values && 64 * (i / PER16) + (int)lane < left); }, whole, edge, first,
           first + (uint32_t)(64 * VECS * PER16 - 1));
  }

  // Sums of the wavefronts, and the largest keys of their lists: this thread's, and how
  // many of the others are larger.
  LogprobPart part = {w.m, wave_sum(w.s), wave_sum(w.t), w.before};
  uint64_t key = 0;
  int above = (int)lane;   // (lists are sorted)
  const uint32_t me = ROW_WAVES == 1 ? lane : tid;
  static_assert(kTop <= 64, "a lane a key");
  for (bool joined = false;; joined = true) {
    if (a.top) w.best.cut();
    key = 0;
    above = (int)lane;
    if ((int)lane < w.best.n) key = w.best.list[lane];
    if (ROW_WAVES == 1) break;
    if (lane == 0) {
      wave_part[wave] = part;
      counts[wave] = w.best.n;
    }
    __syncthreads();
    part = wave_part[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) join(part, wave_part[i]);
    if (key) {   // of each of the others, by halving
      int lo[kWaves - 1], n[kWaves - 1];
#pragma unroll
      for (int i = 0; i < kWaves - 1; ++i) {
        lo[i] = 0;
        n[i] = counts[(wave + 1 + i) % kWaves];
      }
#pragma unroll
      for (int d = kTop; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < kWaves - 1; ++i)
          if (lo[i] + d <= n[i] && lists[(wave + 1 + i) % kWaves][lo[i] + d - 1] > key) lo[i] += d;
#pragma unroll
      for (int i = 0; i < kWaves - 1; ++i) above += lo[i];
    }
    if (joined || a.splits == 1) break;

    // This part for the workgroup that finishes the row: device-scope stores, waited for
    // before the count, and read by device-scope loads.
    uint64_t* const keys = a.keys + (row * a.splits + split) * a.top;
    if (key && above < a.top) __hip_atomic_store(keys + above, key, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    int held = 0;
    for (int i = 0; i < kWaves; ++i) held += counts[i];
    if ((int)tid >= held && (int)tid < a.top) __hip_atomic_store(keys + tid, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (tid == 0) {
      uint64_t* const p = reinterpret_cast<uint64_t*>(a.parts + row * a.splits + split);
      const u32x4 u = __builtin_bit_cast(u32x4, part);
      __hip_atomic_store(p, (uint64_t)u.y << 32 | u.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(p + 1, (uint64_t)u.w << 32 | u.z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __builtin_amdgcn_s_waitcnt(VBQ_VMCNT_IMM(0));
    __syncthreads();
    if (tid == 0) {
      last = __hip_atomic_fetch_add(a.counters + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(a.splits - 1);
      if (last) __hip_atomic_store(a.counters + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!last) return;
    // Each wavefront takes a fourth of the parts' keys and sums, and the four are joined as
    // before. Where there are as many parts as keys wanted, the top-th largest of the
    // parts' own best is a bound that few others pass.
    constexpr int LOADS = kLogprobSplits / kWaves * kTop / 64;
    static_assert(kLogprobSplits <= 64, "a lane a part");
    const int share = (a.splits + kWaves - 1) / kWaves, p0 = wave * share;
    const int mine = min(max(a.splits - p0, 0), share);   // parts p0 .. p0 + mine - 1
    const uint64_t* const from = a.keys + row * a.splits * a.top;
    uint64_t k[LOADS], best = 0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      k[i] = 0;
      if (64 * i + (int)lane < mine * a.top)
        k[i] = __hip_atomic_load(from + p0 * a.top + 64 * i + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const bool bounded = a.top && a.splits >= a.top;
    if (bounded && (int)lane < a.splits) best = __hip_atomic_load(from + lane * a.top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    LogprobPart q = {-__FLT_MAX__, 0.f, 0.f, 0};
    if ((int)lane < mine) {
      const uint64_t* const p = reinterpret_cast<const uint64_t*>(a.parts + row * a.splits + p0 + lane);
      const uint64_t u = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint64_t v = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      q = __builtin_bit_cast(LogprobPart, (u32x4{(uint32_t)u, (uint32_t)(u >> 32), (uint32_t)v, (uint32_t)(v >> 32)}));
    }
    w.best.n = w.best.sorted = 0;
    w.best.least = 0;
    if (bounded) {
      int others = 0;
      for (int i = 0; i < a.splits; i += 8)
#pragma unroll
        for (int c = 0; c < 8; ++c) others += lane_key(best, i + c) > best;
      const uint64_t who = __ballot(best && others == a.top - 1);
      if (who) w.best.least = lane_key(best, __builtin_ctzll(who)) - 1;
    }
#pragma unroll 1
    for (int i = 0; 64 * i < mine * a.top; ++i) {
      uint64_t o = k[0];
#pragma unroll
      for (int c = 1; c < LOADS; ++c) o = i == c ? k[c] : o;
      w.best.offer(o);
    }
    const float m = wave_max(q.m), d = down(q.m, m), f = __builtin_amdgcn_exp2f(d);
    part = {m, wave_sum(f * q.s), wave_sum(f * __builtin_fmaf(d, q.s, q.t)), (int)wave_total((uint32_t)q.before)};
  }

  // Answers. A sum that is no number: the row holds a NaN or an infinity above all.
  const bool bad = part.s != part.s, none = part.s == 0.f;
  const float log_s = log2f(part.s);
  auto logprob = [&](float v) {
    if (none) return -__builtin_inff();
    const bool whole = is_far(part.m) || !(fabsf(v) < 0x1p100f);   // (beyond, what log s holds of b's rounding is nothing)
    return whole ? (v - part.m) - log_s * kLn2 : (__builtin_fmaf(v, kLog2e, -to_base(part.m)) - log_s) * kLn2;
  };
  if (me == 0) {
    const float nan = __builtin_nanf("");
    if (a.lse) a.lse[row] = bad ? nan : none ? -__builtin_inff() : __builtin_fmaf(log_s, kLn2, part.m);
    if (a.entropy) a.entropy[row] = bad ? nan : none ? 0.f : (log_s - part.t / part.s) * kLn2;
    if (a.tokens) {
      const bool there = w.count && !bad;
      a.logprob[row] = there ? logprob(w.given) : nan;
      a.rank[row] = there ? part.before : -1;
    }
  }
  if (bad) {
    if ((int)me < a.top) {
      a.top_logprob[row * a.top + me] = __builtin_nanf("");
      a.top_index[row * a.top + me] = -1;
    }
  } else if (key && above < a.top) {
    a.top_logprob[row * a.top + above] = logprob(key_value(key));
    a.top_index[row * a.top + above] = (int32_t)key_index(key);
  }
}

}  // namespace

// Workgroups of a row: as many as there are steps for, where rows alone leave places on
// the chip (more than one for as many rows as there are counters, at most).
int logprob_splits(int rows, int vocab) {
  const int64_t steps = ((int64_t)vocab + kLogprobStep - 1) / kLogprobStep, most = (steps + kWaves - 1) / kWaves;
  int64_t n = 2 * VBQ_LOGPROBS_COUNTERS / rows;
  n = n < most ? n : most;
  return (int)(n < 1 ? 1 : n < kLogprobSplits ? n : kLogprobSplits);
}

template <int ROW_WAVES>
static hipError_t launch(const Logprobs& a, int dtype, int64_t groups, hipStream_t s) {
  if (groups * (64 * kWaves) > (int64_t)UINT32_MAX) return hipErrorNotSupported;
  const dim3 grid((uint32_t)groups);
  if (dtype == VBQ_F16) k_token_logprobs<VBQ_F16, ROW_WAVES><<<grid, 64 * kWaves, 0, s>>>(a);
  else if (dtype == VBQ_BF16) k_token_logprobs<VBQ_BF16, ROW_WAVES><<<grid, 64 * kWaves, 0, s>>>(a);
  else k_token_logprobs<VBQ_F32, ROW_WAVES><<<grid, 64 * kWaves, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_token_logprobs(const Logprobs& a, int dtype, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (a.splits == 1 && a.vocab <= kLogprobStep * 2) return launch<1>(a, dtype, ((int64_t)a.rows + kWaves - 1) / kWaves, s);
  return launch<kWaves>(a, dtype, (int64_t)a.rows * a.splits, s);
}

}  // namespace vbq
