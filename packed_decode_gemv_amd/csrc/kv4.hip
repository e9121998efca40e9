// The 4-bit key/value cache: quantising tokens as they are written, and
// reading them back. The layout and the quantiser are stated in vbq.h.
//
// One wavefront takes eight consecutive tokens (an octet: the tokens whose
// value codes share words) of one head. Lane l = token + 8 * e holds channels
// 8e .. 8e+7 of each group of one token: 16 bytes of fp16 per load, a group's
// minimum and maximum over three exchanges (lanes 8, 16, 32 apart), and one
// word of eight codes. For keys that word is a word of the cache; for values
// the eight lanes of a channel octet transpose their 8x8 nibbles in three
// exchanges (lanes 1, 2, 4 apart) and each then holds eight tokens of one
// channel, a word of the cache. Words of an octet that is not written whole
// keep the other tokens' nibbles (one wavefront owns an octet, so the read and
// the write do not race).
#include "kv4.h"

namespace vbq {
namespace {

constexpr float kClamp = 61440.f;

template <int DT>
__device__ inline void load8(const void* base, int64_t elem, float (&x)[8]) {
  if constexpr (DT == VBQ_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == VBQ_F16) {
        const uint32_t u = w[i];   // (bit casts take no vector elements)
        const half2_t h = __builtin_bit_cast(half2_t, u);
        x[2 * i] = (float)h.x;
        x[2 * i + 1] = (float)h.y;
      } else {
        x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
        x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
      }
    }
  }
}

__device__ inline uint32_t bf16_bits(float v) {   // round to nearest even; v is finite
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

template <int DT>
__device__ inline void store8(void* base, int64_t elem, const float (&x)[8]) {
  if constexpr (DT == VBQ_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == VBQ_F16) {
        const half2_t h = {(_Float16)x[2 * i], (_Float16)x[2 * i + 1]};
        w[i] = __builtin_bit_cast(uint32_t, h);
      } else {
        w[i] = bf16_bits(x[2 * i]) | (bf16_bits(x[2 * i + 1]) << 16);
      }
    }
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + elem) = w;
  }
}

// Transposes the 8x8 nibbles that eight lanes (tok = 0..7) hold: nibble n of
// lane t becomes nibble t of lane n.
__device__ inline uint32_t transpose8(uint32_t w, uint32_t tok) {
  const uint32_t p1 = (uint32_t)__shfl_xor((int)w, 1, 64);
  w = (tok & 1u) ? ((w & 0xF0F0F0F0u) | ((p1 >> 4) & 0x0F0F0F0Fu)) : ((w & 0x0F0F0F0Fu) | ((p1 << 4) & 0xF0F0F0F0u));
  const uint32_t p2 = (uint32_t)__shfl_xor((int)w, 2, 64);
  w = (tok & 2u) ? ((w & 0xFF00FF00u) | ((p2 >> 8) & 0x00FF00FFu)) : ((w & 0x00FF00FFu) | ((p2 << 8) & 0xFF00FF00u));
  const uint32_t p4 = (uint32_t)__shfl_xor((int)w, 4, 64);
  return (tok & 4u) ? ((w & 0xFFFF0000u) | (p4 >> 16)) : ((w & 0x0000FFFFu) | (p4 << 16));
}

// One octet of one head of one sequence.
struct Octet {
  int32_t row0;      // tensor row of the octet's token 0 (may lie before the range)
  uint32_t valid;    // bit t: token t is in the range and its place exists
  uint32_t wanted;   // bit t: token t is in the range
  uint8_t* block;    // null: no page
  uint32_t oct;      // octet in the block, 0..3
};

__device__ inline bool find_octet(const KvCache& c, const KvRange& r, int G, int b, int64_t o, int head, bool report,
                                  Octet& t) {
  const int32_t c0 = r.cu[b], c1 = r.cu[b + 1], s0 = r.start[b];
  const int64_t n = (int64_t)c1 - c0;
  if (c0 < 0 || n < 0 || c1 > r.total || n > r.max_tokens || s0 < 0 || s0 > INT32_MAX - n) {
    if (report) kv_flag(c, VBQ_KV4_FLAG_LENGTH);
    return false;
  }
  const int64_t first = ((int64_t)(s0 >> 3) + o) * 8;   // the octet's first position
  if (n == 0 || first >= (int64_t)s0 + n) return false;
  const int lo = first < s0 ? (int)(s0 - first) : 0;
  const int64_t left = (int64_t)s0 + n - first;
  const int hi = left < 8 ? (int)left : 8;
  t.wanted = (uint32_t)((1u << hi) - (1u << lo)) & 0xFFu;
  t.valid = t.wanted;
  t.row0 = (int32_t)(c0 + (first - s0));
  t.oct = (uint32_t)(first >> 3) & 3u;
  t.block = nullptr;
  const int64_t blk = first >> 5, entry = blk >> c.block_shift;
  if (entry >= r.width) {
    if (report) kv_flag(c, VBQ_KV4_FLAG_LENGTH);
    t.valid = 0;
    return true;
  }
  const int32_t page = r.table[(int64_t)b * r.width + entry];
  if ((uint32_t)page >= (uint32_t)c.n_pages) {
    if (report) kv_flag(c, VBQ_KV4_FLAG_PAGE);
    t.valid = 0;
    return true;
  }
  t.block = kv_block(c, G, (uint32_t)page, head, (uint32_t)blk & ((1u << c.block_shift) - 1u));
  return true;
}

template <int G, int DT>
__global__ __launch_bounds__(256) void k_kv4_append(KvCache c, KvRange r, const void* k, const void* v, int64_t k_ts,
                                                    int64_t k_hs, int64_t v_ts, int64_t v_hs, int64_t octets) {
  const uint32_t lane = threadIdx.x & 63u, tok = lane & 7u, e = lane >> 3;
  const int64_t task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t o = task / c.heads;
  const int head = (int)(task - o * c.heads);
  if (o >= octets) return;
  Octet t;
  if (!find_octet(c, r, G, blockIdx.y, o, head, lane == 0, t) || !t.valid) return;
  const bool mine = (t.valid >> tok) & 1u;
  float x[2][G][8];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t at = (int64_t)(t.row0 + (int)tok) * (kv ? v_ts : k_ts) + head * (kv ? v_hs : k_hs) + 64 * g + 8 * e;
      if (mine) load8<DT>(kv ? v : k, at, x[kv][g]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) x[kv][g][i] = 0.f;
    }
  // Old words of a value octet that is written in part.
  uint32_t keep = 0;   // nibbles that stay
#pragma unroll
  for (int i = 0; i < 8; ++i) keep |= ((t.valid >> i) & 1u) ? 0u : 0xFu << (4 * i);
  uint32_t* const vword = reinterpret_cast<uint32_t*>(t.block + kv_value_codes(G)) + 64 * t.oct + 8 * e + tok;
  uint32_t old[G];
#pragma unroll
  for (int g = 0; g < G; ++g) old[g] = keep ? vword[256 * g] : 0u;
  bool nan = false;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float(&w)[8] = x[kv][g];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool bad = w[i] != w[i];
        nan |= bad;
        w[i] = bad ? 0.f : fminf(fmaxf(w[i], -kClamp), kClamp);
      }
      float lo = w[0], hi = w[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, w[i]);
        hi = fmaxf(hi, w[i]);
      }
#pragma unroll
      for (int d = 8; d < 64; d <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, d, 64));
        hi = fmaxf(hi, __shfl_xor(hi, d, 64));
      }
      const _Float16 s16 = (_Float16)__fdiv_rn(__fsub_rn(hi, lo), 15.f);
      const _Float16 o16 = (_Float16)lo;
      const float s = (float)s16, of = (float)o16;
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = s != 0.f ? fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(w[i], of), s)), 0.f), 15.f) : 0.f;
        word |= (uint32_t)q << (4 * i);
      }
      _Float16* so = reinterpret_cast<_Float16*>(t.block + (kv ? kv_value_so(G) : kv_key_so(G)) + 128 * g);
      const uint32_t place = 8 * t.oct + (kv ? 2 * (tok & 3u) + (tok >> 2) : tok);
      if (mine && e == 0) {
        so[place] = s16;
        so[place + 32] = o16;
      }
      if (kv == 0) {
        uint32_t* kw = reinterpret_cast<uint32_t*>(t.block) + 256 * g;
        if (mine) kw[4 * (16 * (e & 3u) + 4 * t.oct + (tok & 3u)) + 2 * (tok >> 2) + (e >> 2)] = word;
      } else {
        vword[256 * g] = (transpose8(word, tok) & ~keep) | (old[g] & keep);
      }
    }
  if (__ballot(nan && mine) && lane == 0) kv_flag(c, VBQ_KV4_FLAG_NAN);
}

template <int G, int DT>
__global__ __launch_bounds__(256) void k_kv4_read(KvCache c, KvRange r, void* k, void* v, int64_t octets) {
  const uint32_t lane = threadIdx.x & 63u, tok = lane & 7u, e = lane >> 3;
  const int64_t task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t o = task / c.heads;
  const int head = (int)(task - o * c.heads);
  if (o >= octets) return;
  Octet t;
  if (!find_octet(c, r, G, blockIdx.y, o, head, lane == 0, t)) return;
  const bool mine = (t.wanted >> tok) & 1u;
  const bool held = t.valid != 0;
  uint32_t word[2][G];
  _Float16 s16[2][G], o16[2][G];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      word[kv][g] = 0;
      s16[kv][g] = o16[kv][g] = (_Float16)0.f;
      if (!held || !(kv ? v : k)) continue;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(t.block + (kv ? kv_value_codes(G) : 0)) + 256 * g;
      word[kv][g] = kv ? w[64 * t.oct + 8 * e + tok]
                       : w[4 * (16 * (e & 3u) + 4 * t.oct + (tok & 3u)) + 2 * (tok >> 2) + (e >> 2)];
      const _Float16* so =
          reinterpret_cast<const _Float16*>(t.block + (kv ? kv_value_so(G) : kv_key_so(G)) + 128 * g);
      const uint32_t place = 8 * t.oct + (kv ? 2 * (tok & 3u) + (tok >> 2) : tok);
      s16[kv][g] = so[place];
      o16[kv][g] = so[place + 32];
    }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    void* const out = kv ? v : k;
    if (!out) continue;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t w = kv ? transpose8(word[kv][g], tok) : word[kv][g];
      const float s = (float)s16[kv][g], of = (float)o16[kv][g];
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(s, (float)((w >> (4 * i)) & 15u)), of);
      if (mine) store8<DT>(out, ((int64_t)(t.row0 + (int)tok) * c.heads + head) * (64 * G) + 64 * g + 8 * e, x);
    }
  }
}

// Octets that a sequence of max_tokens tokens can touch, and the grid over
// (octet, head) and sequences; no launch when there is nothing to do.
bool octet_grid(const KvCache& c, const KvRange& r, int64_t* octets, dim3* grid, hipError_t* err) {
  *err = hipSuccess;
  if (r.max_tokens == 0 || r.total == 0) return false;
  *octets = ((int64_t)r.max_tokens + 14) / 8;
  const int64_t wgs = (*octets * c.heads + 3) / 4;
  if (wgs > INT32_MAX) {
    *err = hipErrorNotSupported;
    return false;
  }
  *grid = dim3((uint32_t)wgs, (uint32_t)r.batch);
  return true;
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
  int64_t octets;
  dim3 grid;
  hipError_t err;
  if (!octet_grid(c, r, &octets, &grid, &err)) return err;
#define VBQ_CALL(G, DT) k_kv4_append<G, DT><<<grid, 256, 0, s>>>(c, r, k, v, k_ts, k_hs, v_ts, v_hs, octets)
  VBQ_KV4_BY_TYPE(VBQ_CALL)
#undef VBQ_CALL
  return hipGetLastError();
}

hipError_t launch_kv4_read(const KvCache& c, const KvRange& r, void* k, void* v, int dtype, hipStream_t s) {
  int64_t octets;
  dim3 grid;
  hipError_t err;
  if (!octet_grid(c, r, &octets, &grid, &err)) return err;
#define VBQ_CALL(G, DT) k_kv4_read<G, DT><<<grid, 256, 0, s>>>(c, r, k, v, octets)
  VBQ_KV4_BY_TYPE(VBQ_CALL)
#undef VBQ_CALL
  return hipGetLastError();
}

}  // namespace vbq
