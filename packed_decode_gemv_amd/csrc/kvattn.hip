// Attention over the 4-bit key/value cache (layout and meaning in vbq.h).
//
// Rows are the (query token, query head) pairs that share a key/value head:
// row r of a sequence is query r / ratio, head r % ratio of the group. A
// workgroup of four wavefronts takes one row tile and one piece of the token
// axis; wavefront w takes every fourth block of 32 tokens and keeps its own
// running maximum, sum and output in registers. The wavefronts are joined in
// LDS, the pieces in the workspace by the last workgroup that finishes.
//
// Scores. S^T = K Q^T by 16x16x32 fp16 MFMAs: A is a block's key codes, 16
// tokens by 32 channels of one group, B the queries. A code word holds eight
// channels of a token; masked with 0x000F000F and 0x00F000F0 it is a pair of
// fp16 subnormals c 2^-24 and 16 c 2^-24, exact operands (the queries that
// meet the latter are divided by 16). The group's scale and offset enter in
// fp32: score = sum_g s_g (codes . q)_g + o_g sum_g(q).
// Queries are scaled to a largest magnitude in [2^13, 2^14) per row (a power
// of two, undone in the score), so fp16 holds bf16 queries exactly down to
// 2^-28 of the row's largest.
//
// Output. O^T = V^T P^T by the same MFMA: A is 16 channels by 32 tokens of
// values s c + o in fp16 (codes made exact by an exponent that is subtracted
// again, then one packed multiply-add), B the probabilities as they come out
// of the score MFMA: its result holds tokens 4 q + i of a column (row of the
// problem) in lane quarter q, and the cache orders a block's tokens so that
// those of both 16-token halves are the octet 8 q .. 8 q + 7, which is a value
// word. Probabilities carry a factor 2^15 so that fp16 keeps them normal down
// to 2^-29 of the largest.
#include "kv4.h"

namespace vbq {
namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr float kNoMax = -1e30f;     // running maximum before any token
constexpr float kProbShift = 15.f;   // probabilities are held times 2^15
constexpr int kMaxSplits = 256;

__device__ inline float rows_max(float v) {   // over the four lane quarters of a column
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ inline float rows_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Eight codes of a key word as fp16 subnormals: pairs (n, n + 4), the odd
// pairs times 16.
__device__ inline half8_t key_codes(uint32_t w) {
  u32x4 r;
  r.x = w & 0x000F000Fu;
  r.y = w & 0x00F000F0u;
  const uint32_t h = w >> 8;
  r.z = h & 0x000F000Fu;
  r.w = h & 0x00F000F0u;
  return __builtin_bit_cast(half8_t, r);
}

// Constants of the value decode, opaque to the compiler: with the masks in
// scalar and the exponents in vector registers (w & mask) | exponent is one
// instruction; known constants become two with a literal each.
struct Decode {
  uint32_t m0, m4, ex;
  __device__ Decode() : m0(0x000F000Fu), m4(0x00F000F0u), ex(0x64006400u) {
    asm("" : "+s"(m0));
    asm("" : "+s"(m4));
    asm("" : "+v"(ex));
  }
};

// Eight values s c + o of a value word, pairs (n, n + 4); s and o hold the
// pairs' scales and offsets.
__device__ inline half8_t values(const Decode& dc, uint32_t w, const u32x4& s, const u32x4& o) {
  const half2_t one = {(_Float16)1024.f, (_Float16)1024.f}, sx = {(_Float16)0.0625f, (_Float16)0.0625f},
                sb = {(_Float16)-64.f, (_Float16)-64.f};
  const uint32_t h = w >> 8;
  half2_t c[4];
  c[0] = __builtin_bit_cast(half2_t, (w & dc.m0) | dc.ex) - one;
  c[1] = __builtin_elementwise_fma(__builtin_bit_cast(half2_t, (w & dc.m4) | dc.ex), sx, sb);
  c[2] = __builtin_bit_cast(half2_t, (h & dc.m0) | dc.ex) - one;
  c[3] = __builtin_elementwise_fma(__builtin_bit_cast(half2_t, (h & dc.m4) | dc.ex), sx, sb);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t si = s[i], oi = o[i];   // (bit casts take no vector elements)
    r[i] = __builtin_bit_cast(
        uint32_t, __builtin_elementwise_fma(c[i], __builtin_bit_cast(half2_t, si), __builtin_bit_cast(half2_t, oi)));
  }
  return __builtin_bit_cast(half8_t, r);
}

__device__ inline float half_at(const u32x4& w, int i) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i >> 1] >> (16 * (i & 1))));
}

// A block's copy to LDS, 16 bytes a lane and copy (no registers, so the next
// block is on its way while this one is worked on).
template <int G>
__device__ inline void copy_block(uint32_t lds, const uint8_t* p, uint32_t lane) {
  constexpr int BYTES = kKvGroupBytes * G;
  const u32x4 rsrc = make_rsrc(p, BYTES);
#pragma unroll
  for (int i = 0; i < BYTES / 1024; ++i) dma16(rsrc, lds + 1024 * i, 1024 * i + 16 * lane);
  if (lane < (BYTES % 1024) / 16) dma16(rsrc, lds + BYTES / 1024 * 1024, BYTES / 1024 * 1024 + 16 * lane);
}
__device__ inline u32x4 lds16(const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// The blocks that a row tile looks at: sink blocks 0 .. ns-1, then w0 .. w0+nw-1.
struct Reach {
  int32_t ns, w0, nw;
};
__device__ inline Reach reach(int len, int p_min, int p_max, int window, int sinks) {
  Reach r;
  const int end = min(len, p_max + 1);   // tokens that any row sees end here
  const int blocks = end > 0 ? (end + kKvBlock - 1) / kKvBlock : 0;
  r.ns = 0;
  r.w0 = 0;
  if (window) {
    const int lo = p_min - window + 1;   // first token in any row's window
    r.ns = min((min(sinks, end) + kKvBlock - 1) / kKvBlock, blocks);
    r.ns = max(r.ns, 0);
    r.w0 = lo > 0 ? lo / kKvBlock : 0;
    r.w0 = max(r.w0, r.ns);
  }
  r.nw = max(0, blocks - r.w0);
  return r;
}

constexpr float kLn2 = 0.693147180559945309f;

// Four neighbouring outputs, rounded once to the output type.
__device__ inline void store4(const KvAttn& a, int64_t elem, const f32x4& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = v[i];
    if (a.bf16) {
      const uint32_t u = __builtin_bit_cast(uint32_t, f);
      w[i] = f != f ? 0x7FC0u : (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
    } else {
      w[i] = __builtin_bit_cast(uint16_t, (_Float16)f);
    }
  }
  *reinterpret_cast<u32x2*>(a.out + elem) = u32x2{w[0] | (w[1] << 16), w[2] | (w[3] << 16)};
}

__device__ inline void put2(float* p, float x, float y) {   // device-scope, written through
  const f32x2 v = {x, y};
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline f32x2 get2(const float* p) {
  return __builtin_bit_cast(f32x2, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT));
}

template <int G, int NT>
__global__ __launch_bounds__(256, (G <= 2 && NT == 1) ? 4 : (G * NT <= 4) ? 2 : 1) void k_kv4_attn(KvAttn a) {
  constexpr int D = 64 * G, ROWS = 16 * NT, PITCH = D + 4, BYTES = kKvGroupBytes * G;
  // two blocks a wavefront; afterwards the wavefronts' sums, the pieces' factors and partial sums
  constexpr int SUMS = kWaves * 16 * PITCH * 4, JOIN = 16 * kMaxSplits * 4 + 256 * 16;
  constexpr int AFTER = SUMS > JOIN ? SUMS : JOIN;
  __shared__ __attribute__((aligned(16))) uint8_t ring[kWaves * 2 * BYTES > AFTER ? kWaves * 2 * BYTES : AFTER];
  __shared__ float wml[kWaves][ROWS][2];
  __shared__ uint32_t last;
  float* const buf = reinterpret_cast<float*>(ring);
  f32x4* const share = reinterpret_cast<f32x4*>(ring + 16 * kMaxSplits * 4);
  const uint32_t tid = threadIdx.x, lane = tid & 63u, col = lane & 15u, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  const uint32_t split = blockIdx.x % (uint32_t)a.splits;
  const uint32_t tile = blockIdx.x / (uint32_t)a.splits;
  const int rt = (int)(tile % (uint32_t)a.row_tiles);
  const uint32_t bh = tile / (uint32_t)a.row_tiles;
  const int head = (int)(bh % (uint32_t)a.cache.heads), b = (int)(bh / (uint32_t)a.cache.heads);

  const int c0 = a.cu[b], c1 = a.cu[b + 1], len = a.lens[b];
  const int64_t nq = (int64_t)c1 - c0;
  if (c0 < 0 || nq < 0 || c1 > a.total_q || nq > a.max_q || len < 0 || len > a.max_kv ||
      (int64_t)len > ((int64_t)a.width << (a.cache.block_shift + 5))) {
    if (tid == 0) kv_flag(a.cache, VBQ_KV4_FLAG_LENGTH);
    return;
  }
  const int rows = (int)nq * a.ratio, r0 = rt * ROWS;
  if (r0 >= rows) return;
  const int r1 = min(rows, r0 + ROWS);
  const int first = len - (int)nq;   // position of query 0
  const int p_min = a.causal ? first + r0 / a.ratio : len - 1;
  const int p_max = a.causal ? first + (r1 - 1) / a.ratio : len - 1;
  const Reach re = reach(len, p_min, p_max, a.window, a.sinks);
  const int blocks = re.ns + re.nw;
  const int splits = min(a.splits, max(1, (blocks + a.chunk - 1) / a.chunk));   // that have work
  if ((int)split >= splits) return;
  const int i0 = (int)split * a.chunk, i1 = (int)split == splits - 1 ? blocks : i0 + a.chunk;

  // This wavefront's blocks, and the first one's copy.
  const uint32_t in_page = (1u << a.cache.block_shift) - 1u;
  uint8_t* const mine = ring + wave * 2 * BYTES;
  const uint32_t mine_lds = lds_addr(mine);
  int pages = -1;   // lane i: the page of the wavefront's block i (of 64 at a time)
  auto block_of = [&](int idx) { return idx < re.ns ? idx : idx - re.ns + re.w0; };
  // starts the copy of block `it` (number idx of the tile's) and returns whether there is one
  auto start_copy = [&](int it, int idx) {
    if ((it & 63) == 0) {
      const int next = idx + kWaves * (int)lane;
      pages = -1;
      if (next < i1) {
        pages = a.table[(int64_t)b * a.width + (block_of(next) >> a.cache.block_shift)];
        if ((uint32_t)pages >= (uint32_t)a.cache.n_pages) {
          pages = -1;
          kv_flag(a.cache, VBQ_KV4_FLAG_PAGE);
        }
      }
    }
    const int page = __builtin_amdgcn_readlane(pages, it & 63);
    if (page < 0) return false;
    copy_block<G>(mine_lds + (it & 1) * BYTES,
                  kv_block(a.cache, G, (uint32_t)page, head, (uint32_t)block_of(idx) & in_page), lane);
    return true;
  };
  bool have = i0 + wave < i1 && start_copy(0, i0 + wave);

  // Queries: B operands per group and 32-channel step, their sums per group,
  // and what each lane's column sees.
  half8_t qf[NT][G][2];
  float qsum[NT][G], to_log2[NT];
  int hi[NT], lo[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 16 * nt + (int)col;
    const bool in = r < rows;
    const int qi = r / a.ratio, hh = r - qi * a.ratio;
    float x[G][2][8];
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        u32x4 w = {0, 0, 0, 0};
        if (in)
          w = *reinterpret_cast<const u32x4*>(a.q + (int64_t)(c0 + qi) * a.q_ts +
                                              (int64_t)(head * a.ratio + hh) * a.q_hs + 64 * g + 32 * st +
                                              8 * quarter);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
          x[g][st][i] = a.bf16 ? __builtin_bit_cast(float, u << 16)
                               : (float)__builtin_bit_cast(_Float16, (uint16_t)u);
          top = fmaxf(top, fabsf(x[g][st][i]));
        }
      }
    top = rows_max(top);
    int ex = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
    ex = top > 0.f ? max(ex, -100) : 13;
    const float up = ldexpf(1.f, 13 - ex);
    to_log2[nt] = a.scale_log2 * ldexpf(1.f, ex - 13 + 24);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const _Float16 v0 = (_Float16)(x[g][st][i] * up), v1 = (_Float16)(x[g][st][i + 4] * up);
          sum += (float)v0 + (float)v1;
          const _Float16 f = (i & 1) ? (_Float16)0.0625f : (_Float16)1.f;
          qf[nt][g][st][2 * i] = v0 * f;
          qf[nt][g][st][2 * i + 1] = v1 * f;
        }
      qsum[nt][g] = rows_sum(sum) * 0x1p-24f;
    }
    const int p = a.causal ? first + qi : len - 1;
    hi[nt] = in ? min(p, len - 1) : -1;
    lo[nt] = a.window ? p - a.window + 1 : INT32_MIN;
  }

  const Decode dc;
  float m[NT], l[NT];
  f32x4 acc[NT][G][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = kNoMax;
    l[nt] = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int w = 0; w < 4; ++w) acc[nt][g][w] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  for (int it = 0, idx = i0 + wave; idx < i1; ++it, idx += kWaves) {
    const bool here = have;
    // This block's copy has landed, and the last block's reads of the other buffer are done.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    have = idx + kWaves < i1 && start_copy(it + 1, idx + kWaves);
    if (!here) continue;
    const int blk = block_of(idx);
    const uint8_t* const k = mine + (it & 1) * BYTES;

    // scores of the lane's column: token 8 quarter + 4 half + i
    f32x4 sc[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const u32x4 kc = lds16(k + 1024 * g + 16 * lane);
      const u32x4 ks = lds16(k + kv_key_so(G) + 128 * g + 16 * quarter);
      const u32x4 ko = lds16(k + kv_key_so(G) + 128 * g + 64 + 16 * quarter);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const half8_t a0 = key_codes(kc[2 * hf]), a1 = key_codes(kc[2 * hf + 1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f32x4 d = f32x4{0.f, 0.f, 0.f, 0.f};
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, qf[nt][g][0], d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, qf[nt][g][1], d, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sc[nt][hf][i] = __builtin_fmaf(half_at(ks, 4 * hf + i), d[i],
                                           __builtin_fmaf(half_at(ko, 4 * hf + i), qsum[nt][g], sc[nt][hf][i]));
        }
      }
    }
    const int t0 = blk * kKvBlock;
    const bool edge = t0 + kKvBlock - 1 > min(p_min, len - 1) ||
                      (a.window && t0 <= p_max - a.window && t0 + kKvBlock > a.sinks);
    if (edge) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 8 * (int)quarter + 4 * hf + i;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const bool see = t <= hi[nt] && (t >= lo[nt] || t < a.sinks);
            sc[nt][hf][i] = see ? sc[nt][hf][i] : -__builtin_inff();
          }
        }
    }
    // running maximum and sum
    half8_t pf[NT], pl[NT];   // probabilities, and what their rounding to fp16 leaves
    bool grow = false;
    float mt[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float t = -__builtin_inff();
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int i = 0; i < 4; ++i) t = fmaxf(t, sc[nt][hf][i]);
      mt[nt] = fmaxf(m[nt], rows_max(t) * to_log2[nt]);
      grow |= mt[nt] > m[nt];
    }
    if (__any(grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float f = __builtin_amdgcn_exp2f(m[nt] - mt[nt]);
        m[nt] = mt[nt];
        l[nt] *= f;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int w = 0; w < 4; ++w) acc[nt][g][w] *= f;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float base = kProbShift - m[nt];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[nt][0][i], to_log2[nt], base));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[nt][1][i], to_log2[nt], base));
        l[nt] += p0 + p1;
        pf[nt][2 * i] = (_Float16)p0;
        pf[nt][2 * i + 1] = (_Float16)p1;
        pl[nt][2 * i] = (_Float16)(p0 - (float)pf[nt][2 * i]);
        pl[nt][2 * i + 1] = (_Float16)(p1 - (float)pf[nt][2 * i + 1]);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const u32x4 vc = lds16(k + kv_value_codes(G) + 1024 * g + 16 * lane);
      u32x4 vs = lds16(k + kv_value_so(G) + 128 * g + 16 * quarter);
      u32x4 vo = lds16(k + kv_value_so(G) + 128 * g + 64 + 16 * quarter);
      if (t0 + kKvBlock > len) {   // places past the sequence's end may hold anything
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 8 * (int)quarter + i;
          const uint32_t keep = t + 4 < len ? 0xFFFFFFFFu : t < len ? 0x0000FFFFu : 0u;
          vs[i] &= keep;
          vo[i] &= keep;
        }
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const half8_t v = values(dc, vc[w], vs, vo);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][g][w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pf[nt], acc[nt][g][w], 0, 0, 0);
          acc[nt][g][w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pl[nt], acc[nt][g][w], 0, 0, 0);
        }
      }
    }
  }

  // Join the four wavefronts: every one scales its sums to the common maximum.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    l[nt] = rows_sum(l[nt]);
    if (quarter == 0) {
      wml[wave][16 * nt + col][0] = m[nt];
      wml[wave][16 * nt + col][1] = l[nt];
    }
  }
  __syncthreads();
  const bool whole = splits == 1;
  float* const pacc = a.acc + ((size_t)tile * a.splits + split) * ROWS * D;
  float* const pml = a.ml + ((size_t)tile * a.splits + split) * ROWS * 2;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (r0 + 16 * nt >= rows) break;
    if (nt) __syncthreads();   // the buffer is taken again
    {
      const int rr = 16 * nt + (int)col;
      float top = wml[0][rr][0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, wml[w][rr][0]);
      const float f = __builtin_amdgcn_exp2f(m[nt] - top);
      float* const mine = buf + (wave * 16 + col) * PITCH + 16 * quarter;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 v = {acc[nt][g][0][i] * f, acc[nt][g][1][i] * f, acc[nt][g][2][i] * f, acc[nt][g][3][i] * f};
          *reinterpret_cast<f32x4*>(mine + 64 * g + 4 * i) = v;
        }
    }
    __syncthreads();
    for (int e = (int)tid; e < 16 * (D / 4); e += 256) {
      const int row = e / (D / 4), c = e % (D / 4), rr = 16 * nt + row;
      if (r0 + rr >= rows) break;
      float top = wml[0][rr][0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, wml[w][rr][0]);
      float sum = 0.f;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        sum += wml[w][rr][1] * __builtin_amdgcn_exp2f(wml[w][rr][0] - top);
        v += *reinterpret_cast<const f32x4*>(buf + (w * 16 + row) * PITCH + 4 * c);
      }
      if (whole) {
        const int r = r0 + rr, qi = r / a.ratio, hh = r - qi * a.ratio;
        const int64_t o = (int64_t)(c0 + qi) * a.n_heads + head * a.ratio + hh;
        const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
        store4(a, o * D + 4 * c, v * inv);
        if (a.lse && c == 0) a.lse[o] = (top + __builtin_amdgcn_logf(sum) - kProbShift) * kLn2;
      } else {
        float* const d = pacc + (size_t)rr * D + 4 * c;
        put2(d, v[0], v[1]);
        put2(d + 2, v[2], v[3]);
        if (c == 0) put2(pml + 2 * rr, top, sum);
      }
    }
  }
  if (whole) return;

  // Join the pieces. The sums above are device-scope stores, which write
  // through the caches; each wavefront waits for its own before the barrier,
  // so when the counter counts this piece its sums can be read by every
  // workgroup's device-scope loads. The last piece adds all of them in order.
  __builtin_amdgcn_s_waitcnt(VBQ_VMCNT_IMM(0));
  __syncthreads();
  if (tid == 0)
    last = __hip_atomic_fetch_add(&a.counters[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
           (uint32_t)(splits - 1);
  __syncthreads();
  if (!last) return;
  if (tid == 0) __hip_atomic_store(&a.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const float* const tacc = a.acc + (size_t)tile * a.splits * ROWS * D;
  const float* const tml = a.ml + (size_t)tile * a.splits * ROWS * 2;
#pragma unroll 1
  for (int nt = 0; nt < NT; ++nt) {
    const int nrow = min(16, rows - r0 - 16 * nt);
    if (nrow <= 0) break;
    __syncthreads();
    {   // sixteen lanes a row: the common maximum, the total, each piece's factor
      const int row = (int)(tid >> 4), j = (int)(tid & 15u);
      float pm[kMaxSplits / 16], pl[kMaxSplits / 16];
      float top = kNoMax;
#pragma unroll
      for (int i = 0; i < kMaxSplits / 16; ++i) {
        const int sp = 16 * i + j;
        pm[i] = kNoMax;
        pl[i] = 0.f;
        if (row < nrow && sp < splits) {
          const f32x2 v = get2(tml + ((size_t)sp * ROWS + 16 * nt + row) * 2);
          pm[i] = v.x;
          pl[i] = v.y;
        }
        top = fmaxf(top, pm[i]);
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 16));
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxSplits / 16; ++i) {
        const int sp = 16 * i + j;
        const float f = __builtin_amdgcn_exp2f(pm[i] - top);
        sum += pl[i] * f;
        if (sp < splits) buf[row * kMaxSplits + sp] = f;
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor(sum, d, 16);
      if (j == 0) {
        wml[0][row][0] = top;
        wml[0][row][1] = sum;
      }
    }
    __syncthreads();
    // Threads beyond the rows' outputs share the pieces.
    const int ne = nrow * (D / 4), parts = ne <= 128 ? 256 / ne : 1;
    for (int e0 = 0; e0 < ne; e0 += 256) {
      const int e = parts > 1 ? (int)tid % ne : e0 + (int)tid, part = parts > 1 ? (int)tid / ne : 0;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      const int row = e / (D / 4), c = e % (D / 4);
      if (e < ne && part < parts) {
        const float* p = tacc + (size_t)(16 * nt + row) * D + 4 * c;
        const float* w = buf + row * kMaxSplits;
#pragma unroll 8
        for (int sp = part; sp < splits; sp += parts) {
          const float* u = p + (size_t)sp * ROWS * D;
          const f32x2 x = get2(u), y = get2(u + 2);
          v += f32x4{x.x, x.y, y.x, y.y} * w[sp];
        }
      }
      if (parts > 1) {
        share[tid] = v;
        __syncthreads();
        if (part == 0)
          for (int i = 1; i < parts; ++i) v += share[e + i * ne];
      }
      if (e < ne && part == 0) {
        const int r = r0 + 16 * nt + row, qi = r / a.ratio, hh = r - qi * a.ratio;
        const int64_t o = (int64_t)(c0 + qi) * a.n_heads + head * a.ratio + hh;
        const float top = wml[0][row][0], sum = wml[0][row][1];
        const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
        store4(a, o * D + 4 * c, v * inv);
        if (a.lse && c == 0) a.lse[o] = (top + __builtin_amdgcn_logf(sum) - kProbShift) * kLn2;
      }
    }
  }
}

}  // namespace

KvAttnPlan kv4_attn_plan(int batch, int heads, int ratio, int groups, int max_q, int max_kv, int window, int sinks) {
  KvAttnPlan p;
  const int64_t rows = (int64_t)max_q * ratio;
  p.rows = rows <= 16 ? 16 : 32;
  p.row_tiles = rows > 0 ? (int32_t)((rows + p.rows - 1) / p.rows) : 1;
  p.tiles = (int64_t)batch * heads * p.row_tiles;
  int64_t blocks = ((int64_t)max_kv + kKvBlock - 1) / kKvBlock;
  if (window) {   // a row tile sees its sinks, its queries' windows and the blocks these end in
    const int64_t reach = ((int64_t)sinks + kKvBlock - 1) / kKvBlock +
                          ((int64_t)window + (p.rows + ratio - 1) / ratio) / kKvBlock + 2;
    blocks = blocks < reach ? blocks : reach;
  }
  // Pieces: enough workgroups for four on every CU, none under two blocks a wavefront.
  int64_t splits = (1024 + p.tiles - 1) / p.tiles;
  const int64_t most = (blocks + 2 * kWaves - 1) / (2 * kWaves);
  splits = splits < most ? splits : most;
  splits = splits < kMaxSplits ? splits : kMaxSplits;
  if (p.tiles > VBQ_KV4_COUNTER_BYTES / 4 || splits < 1) splits = 1;
  int64_t chunk = (blocks + splits - 1) / splits;
  chunk = (chunk + kWaves - 1) / kWaves * kWaves;
  p.chunk = (int32_t)(chunk < 1 ? kWaves : chunk);
  p.splits = (int32_t)((blocks + p.chunk - 1) / p.chunk);
  if (p.splits < 1) p.splits = 1;
  return p;
}

hipError_t launch_kv4_attention(const KvAttn& a, const KvAttnPlan& p, int batch, hipStream_t s) {
  const int64_t wgs = p.tiles * p.splits;
  if (wgs > INT32_MAX) return hipErrorNotSupported;
  const dim3 grid((uint32_t)wgs);
#define VBQ_CALL(G)                                          \
  if (p.rows == 16) k_kv4_attn<G, 1><<<grid, 256, 0, s>>>(a); \
  else k_kv4_attn<G, 2><<<grid, 256, 0, s>>>(a)
  switch (a.cache.groups) {
    case 1: VBQ_CALL(1); break;
    case 2: VBQ_CALL(2); break;
    case 3: VBQ_CALL(3); break;
    default: VBQ_CALL(4); break;
  }
#undef VBQ_CALL
  return hipGetLastError();
}

}  // namespace vbq
