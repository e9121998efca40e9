// Norms of queries and keys for each head, with the rotation by position in the
// same pass (meaning in vbq.h).
//
// A head of D = 64 G channels takes 4 G lanes of a wavefront, 16 channels each: two
// chunks of eight that hold whole pairs, so no channel moves between lanes. With
// halves paired, lane e < R / 16 holds channels 8e .. 8e+7 and R/2 + 8e ..; lanes
// beyond, and all lanes where neighbours are paired, hold 16e .. 16e+15. A
// wavefront takes 64 / 4G heads of one token; the token's cosines and sines are worked
// out a pair a lane and read back from LDS. (Two such passes a wavefront save half of
// that, but leave less on its way: 25763 bf16 tokens of 32 + 8 heads of 128 take 98 us by
// one and 96 by two, 7001 fp32 tokens of 16 + 4 heads of 256 43 and 45; five take 105
// and 52.)
//   Memory bounds it: those move 528 and 215 MB, at 5.4 and 5.0 TB/s; a large copy
// reaches 5.1 to 6.2 from card to card.
//
// Angles. position * inv_freq in turns, in binary64: 2^31 positions leave 8e-8 of a
// turn, and what is left of whole turns is rounded to binary32 only then.
#include "vbq_common.h"

#include "heads.h"

namespace vbq {
namespace {

typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
constexpr int kHeadWaves = 4;
constexpr double kTurnsPerRadian = 0.15915494309189533577;

template <int DT>
__device__ inline void load8(const void* base, int64_t elem, float (&x)[8]) {
  if constexpr (DT == VBQ_F32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + elem);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = a[i], w = b[i];
      x[i] = __builtin_bit_cast(float, u);
      x[4 + i] = __builtin_bit_cast(float, w);
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + elem);
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
    }
  }
}

__device__ inline void store8(void* base, int64_t elem, int dt, const float (&x)[8]) {
  if (dt == VBQ_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
    return;
  }
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dt == VBQ_F16) {
      const half2_t h = {(_Float16)x[2 * i], (_Float16)x[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, h);
    } else {
      const bf2_t h = {(__bf16)x[2 * i], (__bf16)x[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, h);
    }
  }
  *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + elem) = w;
}

// Sum over the 4 G lanes of a head, the same in each of them.
template <int G>
__device__ inline float head_sum(float v, uint32_t lane) {
  v += __shfl_xor(v, 1, 64);
  v += __shfl_xor(v, 2, 64);
  if constexpr (G == 2 || G == 4) v += __shfl_xor(v, 4, 64);
  if constexpr (G == 4) v += __shfl_xor(v, 8, 64);
  if constexpr (G == 3) {
    const int first = (int)(lane / 12u * 12u);
    v = (__shfl(v, first, 64) + __shfl(v, first + 4, 64)) + __shfl(v, first + 8, 64);
  }
  return v;
}

template <int G, int DT, bool NEIGHBOURS>
__global__ __launch_bounds__(64 * kHeadWaves) void k_head_norm_rotary(HeadRotary a) {
  constexpr int D = 64 * G, LANES = 4 * G, HEADS = 64 / LANES;   // lanes of a head, heads at a time
  __shared__ __attribute__((aligned(16))) float2 turn[kHeadWaves][D / 2];
  const uint32_t lane = threadIdx.x & 63u;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t task = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kHeadWaves + wave;
  const int64_t token = task / a.passes;
  if (token >= a.tokens) return;
  const int pass = (int)(task - token * a.passes);
  const int e = (int)(lane % LANES), slot = (int)(lane / LANES);

  // The token's turns, a pair a lane.
  const int half = a.rotary_dim / 2;
#pragma unroll
  for (int j = 0; j < (D / 2 + 63) / 64; ++j) {
    const int p = 64 * j + (int)lane;
    if (p < half) {
      const int axis = a.axis ? min((int)a.axis[p], a.axes - 1) : 0;
      const double t = (double)a.positions[axis * a.position_stride + token] * ((double)a.inv_freq[p] * kTurnsPerRadian);
      const float rest = (float)(t - rint(t));
      float s, c;
      sincospif(2.f * rest, &s, &c);
      turn[wave][p] = make_float2(c, s);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

  const bool turned = 16 * e < a.rotary_dim;
  int ch0 = 16 * e, ch1 = 16 * e + 8;   // the lane's chunks
  if (!NEIGHBOURS && turned) {
    ch0 = 8 * e;
    ch1 = half + 8 * e;
  }
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 t = turned ? turn[wave][8 * e + i] : make_float2(1.f, 0.f);
    cs[i] = t.x;
    sn[i] = t.y;
  }

  const int q_passes = (a.q.heads + HEADS - 1) / HEADS;
  const bool is_k = pass >= q_passes;
  const HeadRows& t = is_k ? a.k : a.q;
  const int head = (is_k ? pass - q_passes : pass) * HEADS + slot;
  const bool in = head < t.heads && slot < HEADS;
  float x0[8], x1[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x0[i] = x1[i] = 0.f;
  if (in) {
    const int64_t at = token * t.in_ts + head * t.in_hs;
    load8<DT>(t.in, at + ch0, x0);
    load8<DT>(t.in, at + ch1, x1);
  }
  if (t.weight) {
    float w0[8], w1[8];
    load8<VBQ_F32>(t.weight, ch0, w0);
    load8<VBQ_F32>(t.weight, ch1, w1);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(x0[i], x0[i], __builtin_fmaf(x1[i], x1[i], sum));
    const float r = rsqrtf(__builtin_fmaf(head_sum<G>(sum, lane), 1.f / D, a.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x0[i] *= r * w0[i];
      x1[i] *= r * w1[i];
    }
  }
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& u = NEIGHBOURS ? (i < 4 ? x0[2 * i] : x1[2 * i - 8]) : x0[i];
      float& v = NEIGHBOURS ? (i < 4 ? x0[2 * i + 1] : x1[2 * i - 7]) : x1[i];
      const float y = __builtin_fmaf(u, cs[i], -v * sn[i]);
      v = __builtin_fmaf(v, cs[i], u * sn[i]);
      u = y;
    }
  }
  if (in) {
    const int64_t at = token * t.out_ts + head * t.out_hs;
    store8(t.out, at + ch0, t.out_dtype, x0);
    store8(t.out, at + ch1, t.out_dtype, x1);
  }
}

}  // namespace

hipError_t launch_head_norm_rotary(HeadRotary a, int dtype, hipStream_t s) {
  const int groups = a.head_dim / 64, heads = 64 / (4 * groups);
  const int64_t passes = (a.q.heads + heads - 1) / heads + (a.k.heads + heads - 1) / heads;
  if (a.tokens == 0 || passes == 0) return hipSuccess;
  a.passes = (int32_t)passes;
  const int64_t groups_n = (a.tokens * passes + kHeadWaves - 1) / kHeadWaves;
  // (a dimension holds fewer than 2^32 threads; workgroups past the last token have nothing to do)
  constexpr int64_t ROW = 1 << 23;
  const int64_t across = groups_n < ROW ? groups_n : ROW, down = (groups_n + across - 1) / across;
  if (down > 65535) return hipErrorNotSupported;
  const dim3 grid((uint32_t)across, (uint32_t)down);
#define VBQ_ONE(G, DT)                                                                               \
  if (a.interleaved) k_head_norm_rotary<G, DT, true><<<grid, 64 * kHeadWaves, 0, s>>>(a);            \
  else k_head_norm_rotary<G, DT, false><<<grid, 64 * kHeadWaves, 0, s>>>(a)
#define VBQ_BY_TYPE(G)                       \
  if (dtype == VBQ_F16) { VBQ_ONE(G, VBQ_F16); }      \
  else if (dtype == VBQ_BF16) { VBQ_ONE(G, VBQ_BF16); } \
  else { VBQ_ONE(G, VBQ_F32); }
  switch (groups) {
    case 1: VBQ_BY_TYPE(1); break;
    case 2: VBQ_BY_TYPE(2); break;
    case 3: VBQ_BY_TYPE(3); break;
    default: VBQ_BY_TYPE(4); break;
  }
#undef VBQ_BY_TYPE
#undef VBQ_ONE
  return hipGetLastError();
}

}  // namespace vbq
