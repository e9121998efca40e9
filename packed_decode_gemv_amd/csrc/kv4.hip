// The 4-bit key/value cache: quantising tokens as they are written, and
// reading them back. The layout and the quantiser are stated in vbq.h.
//
// Writing. A workgroup takes a block of 32 tokens of one head (so that the cache
// of one die gathers the lines it writes), a wavefront eight of them (an octet:
// the tokens whose value codes share words). Lane l = token + 8 * e holds
// channels 8e .. 8e+7 of each group of one token: 16 bytes of fp16 per load, a
// group's minimum and maximum over three exchanges (lanes 8, 16, 32 apart), and
// one word of eight codes. For keys that word is a word of the cache; for values
// the eight lanes of a channel octet transpose their 8x8 nibbles in three
// exchanges (lanes 1, 2, 4 apart) and each then holds eight tokens of one
// channel, a word of the cache. Words of an octet that is not written whole
// keep the other tokens' nibbles (one wavefront owns an octet, so the read and
// the write do not race).
//   25800 bf16 tokens of 8 heads of 128 take 44 us, 135 MB at 3.1 TB/s. The
// arithmetic bounds it (about 34 us of vector issue; a plain copy of as many bytes
// takes 22): a correctly rounded quotient a value made it 56 us. Codes are
// decided by t = (w - o) * rcp(s): rcp is within 2^-23 and the product within
// 2^-24, so t is within 16 * 2^-22 = 2^-18 of the correctly rounded quotient
// where a code hangs on it (t < 16), and only a t within 2^-16 of a tie takes
// the division (one wavefront's group in 60).
//
// Reading. One wavefront takes a block of 32 tokens of one head, 16 bytes a lane
// as they lie, so the look-ups are paid once for 32 tokens and nothing moves
// between lanes: a key word is eight channels of a token, the four value words
// of a lane four channels of eight tokens. HBM writes bound it: 65000 bf16
// tokens of 8 heads of 128 take 81 us, 334 MB at 4.1 TB/s, where a copy that
// reads as much as it writes reaches 6.2.
#include "kv4.h"

namespace vbq {
namespace {

constexpr float kClamp = 61440.f;

typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));

// Eight numbers, and whether one is NaN or beyond the clamp (magnitudes order
// like their bits).
template <int DT>
__device__ inline bool load8(const void* base, int64_t elem, float (&x)[8]) {
  if constexpr (DT == VBQ_F32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + elem);
    const u32x4 a = p[0], b = p[1];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = a[i], w = b[i];
      x[i] = __builtin_bit_cast(float, u);
      x[4 + i] = __builtin_bit_cast(float, w);
      top = max(max(top, u << 1), w << 1);
    }
    return top > (__builtin_bit_cast(uint32_t, kClamp) << 1);
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + elem);
    ushort2_t top = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = w[i];
      if constexpr (DT == VBQ_F16) {
        const half2_t h = __builtin_bit_cast(half2_t, u);
        x[2 * i] = (float)h.x;
        x[2 * i + 1] = (float)h.y;
      } else {
        x[2 * i] = __builtin_bit_cast(float, u << 16);
        x[2 * i + 1] = __builtin_bit_cast(float, u & 0xFFFF0000u);
      }
      top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2_t, u & 0x7FFF7FFFu));
    }
    constexpr uint16_t most = DT == VBQ_F16 ? 0x7B80 : 0x4770;   // 61440
    return top.x > most || top.y > most;
  }
}

typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kXor3 = 0x1B, kXor7 = 0x141, kXor8 = 0x128;

// Transposes the 8x8 nibbles that eight lanes (tok = 0..7) hold: nibble n of
// lane t becomes nibble t of lane n.
__device__ inline uint32_t swap_with(uint32_t w, uint32_t other, bool upper, uint32_t upper_mask, int bits) {
  // the half of w that stays, and the other lane's half moved into its place
  const uint32_t keep = upper ? upper_mask : ~upper_mask, turn = upper ? bits : 32 - bits;
  return (w & keep) | (__builtin_amdgcn_alignbit(other, other, turn) & ~keep);
}
__device__ inline uint32_t transpose8(uint32_t w, uint32_t tok) {
  w = swap_with(w, dpp<kXor1>(w), tok & 1u, 0xF0F0F0F0u, 4);
  w = swap_with(w, dpp<kXor2>(w), tok & 2u, 0xFF00FF00u, 8);
  return swap_with(w, dpp<kXor3>(dpp<kXor7>(w)), tok & 4u, 0xFFFF0000u, 16);
}

// Minimum and maximum over the lanes 8, 16 and 32 apart.
__device__ inline float as_float(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ inline uint32_t as_bits(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ inline float min2(float x, float y) { return __builtin_amdgcn_fmed3f(x, y, -__builtin_inff()); }
__device__ inline float max2(float x, float y) { return __builtin_amdgcn_fmed3f(x, y, __builtin_inff()); }
__device__ inline void spread_min_max(float& lo, float& hi) {   // (finite numbers)
  typedef uint32_t pair_t __attribute__((ext_vector_type(2)));
  lo = min2(lo, as_float(dpp<kXor8>(as_bits(lo))));
  hi = max2(hi, as_float(dpp<kXor8>(as_bits(hi))));
  pair_t p = __builtin_amdgcn_permlane16_swap(as_bits(lo), as_bits(lo), false, false);
  pair_t q = __builtin_amdgcn_permlane16_swap(as_bits(hi), as_bits(hi), false, false);
  uint32_t p0 = p.x, p1 = p.y, q0 = q.x, q1 = q.y;
  lo = min2(as_float(p0), as_float(p1));
  hi = max2(as_float(q0), as_float(q1));
  p = __builtin_amdgcn_permlane32_swap(as_bits(lo), as_bits(lo), false, false);
  q = __builtin_amdgcn_permlane32_swap(as_bits(hi), as_bits(hi), false, false);
  p0 = p.x, p1 = p.y, q0 = q.x, q1 = q.y;
  lo = min2(as_float(p0), as_float(p1));
  hi = max2(as_float(q0), as_float(q1));
}

// Numbers of a sequence that fit the call.
__device__ inline bool range_fits(const KvRange& r, int32_t c0, int64_t n, int32_t c1, int32_t s0) {
  return c0 >= 0 && n >= 0 && c1 <= r.total && n <= r.max_tokens && s0 >= 0 && s0 <= INT32_MAX - 64 - n;
}

// The page of a sequence's block, or -1.
__device__ inline int32_t find_page(const KvCache& c, const KvRange& r, int b, int32_t blk, bool report) {
  const int32_t entry = blk >> c.block_shift;
  if (entry >= r.width) {
    if (report) kv_flag(c, VBQ_KV4_FLAG_LENGTH);
    return -1;
  }
  const int32_t page = r.table[(int64_t)b * r.width + entry];
  if ((uint32_t)page < (uint32_t)c.n_pages) return page;
  if (report) kv_flag(c, VBQ_KV4_FLAG_PAGE);
  return -1;
}

template <int G, int DT>
__global__ __launch_bounds__(256) void k_kv4_append(KvCache c, KvRange r, const void* k, const void* v, int64_t k_ts,
                                                    int64_t k_hs, int64_t v_ts, int64_t v_hs) {
  const uint32_t lane = threadIdx.x & 63u, tok = lane & 7u, e = lane >> 3;
  const uint32_t oct = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = (int)(blockIdx.x % (uint32_t)c.heads), b = (int)blockIdx.y;
  const int32_t c0 = r.cu[b], c1 = r.cu[b + 1], s0 = r.start[b];
  const int64_t n = (int64_t)c1 - c0;
  if (!range_fits(r, c0, n, c1, s0)) {
    if (threadIdx.x == 0) kv_flag(c, VBQ_KV4_FLAG_LENGTH);
    return;
  }
  if (n == 0) return;   // (an idle sequence's row of the table may hold anything, another's page too)
  // the octet's first position, and its tokens that are in the range
  const int64_t blk = (s0 >> 5) + (int64_t)(blockIdx.x / (uint32_t)c.heads), first = 32 * blk + 8 * oct;
  const int64_t ahead = (int64_t)s0 + n - first;
  if (ahead <= 0 || first + 8 <= s0) return;
  const int from = first < s0 ? (int)(s0 - first) : 0, to = ahead < 8 ? (int)ahead : 8;
  const uint32_t valid = (uint32_t)((1u << to) - (1u << from)) & 0xFFu;
  const int64_t row0 = c0 + (first - s0);
  const bool mine = (valid >> tok) & 1u;
  float x[2][G][8];
  bool odd = false;   // a NaN, or a number beyond the clamp
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t at = (row0 + tok) * (kv ? v_ts : k_ts) + head * (kv ? v_hs : k_hs) + 64 * g + 8 * e;
      if (mine) odd |= load8<DT>(kv ? v : k, at, x[kv][g]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) x[kv][g][i] = 0.f;
    }
  const int32_t page = find_page(c, r, b, (int32_t)blk, lane == 0);
  if (page < 0) return;
  uint8_t* const block = kv_block(c, G, (uint32_t)page, head, (uint32_t)blk & ((1u << c.block_shift) - 1u));
  // Old words of a value octet that is written in part.
  uint32_t keep = 0;   // nibbles that stay
#pragma unroll
  for (int i = 0; i < 8; ++i) keep |= ((valid >> i) & 1u) ? 0u : 0xFu << (4 * i);
  uint32_t* const vword = reinterpret_cast<uint32_t*>(block + kv_value_codes(G)) + 64 * oct + 8 * e + tok;
  uint32_t old[G];
#pragma unroll
  for (int g = 0; g < G; ++g) old[g] = keep ? vword[256 * g] : 0u;
  if (__any(odd)) {
    bool nan = false;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& w = x[kv][g][i];
          const bool bad = w != w;
          nan |= bad;
          w = bad ? 0.f : __builtin_amdgcn_fmed3f(w, -kClamp, kClamp);
        }
    if (__any(nan) && lane == 0) kv_flag(c, VBQ_KV4_FLAG_NAN);
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float(&w)[8] = x[kv][g];
      float lo = min2(w[0], w[1]), hi = max2(w[0], w[1]);
#pragma unroll
      for (int i = 2; i < 8; ++i) {
        lo = min2(lo, w[i]);
        hi = max2(hi, w[i]);
      }
      spread_min_max(lo, hi);
      float scale = __fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f);
      asm("" : "+v"(scale));   // or product and conversion become one instruction that rounds once
      const _Float16 s16 = (_Float16)scale;
      const _Float16 o16 = (_Float16)lo;
      const float s = (float)s16, of = (float)o16;
      const float r = s != 0.f ? __builtin_amdgcn_rcpf(s) : 0.f;
      float q[8], off = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = __builtin_amdgcn_fmed3f(__fmul_rn(__fsub_rn(w[i], of), r), 0.f, 15.f);
        q[i] = rintf(u);
        off = fmaxf(off, fabsf(__fsub_rn(u, q[i])));
      }
      if (__any(off > 0.5f - 0x1p-16f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          q[i] = s != 0.f ? __builtin_amdgcn_fmed3f(rintf(__fdiv_rn(__fsub_rn(w[i], of), s)), 0.f, 15.f) : 0.f;
      }
      // four codes a half, exact as a float
      const float h0 = __builtin_fmaf(q[3], 4096.f, __builtin_fmaf(q[2], 256.f, __builtin_fmaf(q[1], 16.f, q[0])));
      const float h1 = __builtin_fmaf(q[7], 4096.f, __builtin_fmaf(q[6], 256.f, __builtin_fmaf(q[5], 16.f, q[4])));
      const uint32_t word = (uint32_t)h0 | ((uint32_t)h1 << 16);
      _Float16* so = reinterpret_cast<_Float16*>(block + (kv ? kv_value_so(G) : kv_key_so(G)) + 128 * g);
      const uint32_t place = 8 * oct + (kv ? 2 * (tok & 3u) + (tok >> 2) : tok);
      if (mine && e == 0) {
        so[place] = s16;
        so[place + 32] = o16;
      }
      if (kv == 0) {
        uint32_t* kw = reinterpret_cast<uint32_t*>(block) + 256 * g;
        if (mine) kw[4 * (16 * (e & 3u) + 4 * oct + (tok & 3u)) + 2 * (tok >> 2) + (e >> 2)] = word;
      } else {
        vword[256 * g] = (transpose8(word, tok) & ~keep) | (old[g] & keep);
      }
    }
}

// N neighbouring channels of a row, rounded once.
template <int DT, int N>
__device__ inline void store_row(void* base, int64_t elem, const float (&x)[N]) {
  if constexpr (DT == VBQ_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (DT == VBQ_F16) {
        float u = x[2 * i], v = x[2 * i + 1];
        asm("" : "+v"(u), "+v"(v));   // the fp32 value is rounded, not the sum before it (see k_kv4_append)
        const half2_t h = {(_Float16)u, (_Float16)v};
        w[i] = __builtin_bit_cast(uint32_t, h);
      } else {
        const bf2_t h = {(__bf16)x[2 * i], (__bf16)x[2 * i + 1]};
        w[i] = __builtin_bit_cast(uint32_t, h);
      }
    }
    uint16_t* const p = static_cast<uint16_t*>(base) + elem;
    if constexpr (N == 8) *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
  }
}

template <int G, int DT>
__global__ __launch_bounds__(256) void k_kv4_read(KvCache c, KvRange r, void* k, void* v, int64_t blocks) {
  const uint32_t lane = threadIdx.x & 63u, m = lane & 15u, kq = lane >> 4;
  const int64_t task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t o = task / c.heads;
  const int head = (int)(task - o * c.heads);
  if (o >= blocks) return;
  const int b = (int)blockIdx.y;
  const int32_t c0 = r.cu[b], c1 = r.cu[b + 1], s0 = r.start[b];
  const int64_t n = (int64_t)c1 - c0;
  if (!range_fits(r, c0, n, c1, s0)) {
    if (lane == 0) kv_flag(c, VBQ_KV4_FLAG_LENGTH);
    return;
  }
  const int64_t blk = (s0 >> 5) + o, first = blk * 32;   // the block's first position
  if (n == 0 || first >= (int64_t)s0 + n) return;
  // tokens t of the block with from <= t < to are wanted; token t is row row0 + t
  const int from = first < s0 ? (int)(s0 - first) : 0;
  const int to = (int)((int64_t)s0 + n - first < 32 ? (int64_t)s0 + n - first : 32);
  const int64_t row0 = c0 + (first - s0);
  const int32_t page = find_page(c, r, b, (int32_t)blk, lane == 0);
  const uint8_t* const p =
      kv_block(c, G, page < 0 ? 0u : (uint32_t)page, head, (uint32_t)blk & ((1u << c.block_shift) - 1u));
  u32x4 kw[G], vw[G], vs[G], vo[G];
  _Float16 ks[G][2], ko[G][2];
  const uint32_t tok = 8 * (m >> 2) + (m & 3u);   // of the key words' first half; + 4 for the second
#pragma unroll
  for (int g = 0; g < G; ++g) {
    kw[g] = *reinterpret_cast<const u32x4*>(p + 1024 * g + 16 * lane);
    vw[g] = *reinterpret_cast<const u32x4*>(p + kv_value_codes(G) + 1024 * g + 16 * lane);
    const _Float16* const so = reinterpret_cast<const _Float16*>(p + kv_key_so(G) + 128 * g);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ks[g][u] = so[tok + 4 * u];
      ko[g][u] = so[32 + tok + 4 * u];
    }
    vs[g] = *reinterpret_cast<const u32x4*>(p + kv_value_so(G) + 128 * g + 16 * kq);
    vo[g] = *reinterpret_cast<const u32x4*>(p + kv_value_so(G) + 128 * g + 64 + 16 * kq);
  }
  const int64_t row_elems = (int64_t)c.heads * (64 * G);
  if (k) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = (int)tok + 4 * u;
        if (t < from || t >= to) continue;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const uint32_t w = kw[g][2 * u + st];
          const float s = (float)ks[g][u], of = (float)ko[g][u];
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = page < 0 ? 0.f : __builtin_fmaf(s, (float)((w >> (4 * i)) & 15u), of);
          store_row<DT, 8>(k, (row0 + t) * row_elems + head * (64 * G) + 64 * g + 32 * st + 8 * kq, x);
        }
      }
  }
  if (v) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int n8 = 0; n8 < 8; ++n8) {   // token 8 kq + n8: scale at half n8 / 4 of pair n8 % 4
        const int t = 8 * (int)kq + n8;
        if (t < from || t >= to) continue;
        const uint32_t sw = vs[g][n8 & 3], ow = vo[g][n8 & 3];
        const half2_t sp = __builtin_bit_cast(half2_t, sw), op = __builtin_bit_cast(half2_t, ow);
        const float s = (float)(n8 < 4 ? sp.x : sp.y), of = (float)(n8 < 4 ? op.x : op.y);
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = page < 0 ? 0.f : __builtin_fmaf(s, (float)((vw[g][i] >> (4 * n8)) & 15u), of);
        store_row<DT, 4>(v, (row0 + t) * row_elems + head * (64 * G) + 64 * g + 4 * m, x);
      }
  }
}

// Blocks that a sequence can touch, times the heads; 0 when there is nothing to
// do. No sequence has more tokens than the call.
int64_t block_tasks(const KvCache& c, const KvRange& r) {
  if (r.max_tokens == 0 || r.total == 0) return 0;
  return ((int64_t)(r.max_tokens < r.total ? r.max_tokens : r.total) + 62) / 32 * c.heads;
}

}  // namespace

#define VBQ_KV4_BY_GROUPS(DT, CALL)  \
  switch (c.groups) {                \
    case 1: CALL(1, DT); break;      \
    case 2: CALL(2, DT); break;      \
    case 3: CALL(3, DT); break;      \
    default: CALL(4, DT); break;     \
  }
#define VBQ_KV4_BY_TYPE(CALL)                                    \
  if (dtype == VBQ_F16) { VBQ_KV4_BY_GROUPS(VBQ_F16, CALL) }     \
  else if (dtype == VBQ_BF16) { VBQ_KV4_BY_GROUPS(VBQ_BF16, CALL) } \
  else { VBQ_KV4_BY_GROUPS(VBQ_F32, CALL) }

hipError_t launch_kv4_append(const KvCache& c, const KvRange& r, const void* k, const void* v, int dtype,
                             int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs, hipStream_t s) {
  const int64_t tasks = block_tasks(c, r);   // a workgroup a block: an octet a wavefront
  if (tasks == 0) return hipSuccess;
  if (!kv_grid_fits(tasks, 256)) return hipErrorNotSupported;
  const dim3 grid((uint32_t)tasks, (uint32_t)r.batch);
#define VBQ_CALL(G, DT) k_kv4_append<G, DT><<<grid, 256, 0, s>>>(c, r, k, v, k_ts, k_hs, v_ts, v_hs)
  VBQ_KV4_BY_TYPE(VBQ_CALL)
#undef VBQ_CALL
  return hipGetLastError();
}

hipError_t launch_kv4_read(const KvCache& c, const KvRange& r, void* k, void* v, int dtype, hipStream_t s) {
  const int64_t tasks = block_tasks(c, r), groups = (tasks + 3) / 4;   // a wavefront a block
  if (tasks == 0) return hipSuccess;
  if (!kv_grid_fits(groups, 256)) return hipErrorNotSupported;
  const dim3 grid((uint32_t)groups, (uint32_t)r.batch);
#define VBQ_CALL(G, DT) k_kv4_read<G, DT><<<grid, 256, 0, s>>>(c, r, k, v, tasks / c.heads)
  VBQ_KV4_BY_TYPE(VBQ_CALL)
#undef VBQ_CALL
  return hipGetLastError();
}

}  // namespace vbq
