// Attention of sequences that have their first tokens in common (meaning in vbq.h):
// the kernels for heads of 64 G channels; each kvshared_g*.hip instantiates one G.
//
// One launch takes both kinds of tokens: workgroups over the groups' shared tokens,
// where the rows of all of a group's sequences make the tiles, then workgroups over the
// sequences' own. The first are few and long (a tile is cut into parts along the
// tokens, one or two a CU), the second short, and fill the places that are left (own
// tokens first: 32 sequences over 8192 shared tokens 30.4 against 28.7 us, 6 groups of 16
// with 3 queries 67.9 against 60.7). All
// sums go to the workspace, and a second launch joins a row's and answers it. Where a
// sequence's own rows need the kernel for many rows, the two kinds take a launch each;
// so they do where one workgroup of heads of 256 takes a CU and the own tokens' are more
// than the CUs, as several of those fit a CU by themselves. Together and apart, us, groups of 32
// sequences, 100 own tokens: 4 heads of 256, 2 groups of 8192 shared 56.4 and 57.3, 4 of 8192
// 78.9 and 75.0, 16 of 4096 160 and 133; 8 heads of 128 with 4 rows, 6 of 8192 76.8 and 84.6,
// 16 of 4096 120 and 116, 24 of 2048 130 and 131; of 192 with 2, 8 of 4096 87.4 and 93.9;
// groups of 64, 12 heads of 64, 1 of 8192 20.9 and 27.0, 24 of 2048 169 and 196.
// Small calls are one launch of the kernel for few rows, sequence by sequence.
// Own rows that fill tiles of 128 by themselves make enough of a block, and sums of both kinds
// cost more than the shared blocks again: this and kv4_attention over a table that names the
// shared pages in every row, us, bf16, 32 heads of 128 on 8 (4 rows a query): 64 sequences of 257
// queries behind 512 shared tokens 581 and 327, behind 2048 1097 and 884, behind 8192 3293 and
// 3174; 16 of 64 behind 65536 1453 and 1448; 32 of 40 behind 8192 376 and 359, of 20 152 and 193;
// 64 of 9 148 and 356.
//
// Measured, 32 heads of 128 on 8: 64 sequences over 65000 shared tokens (bf16) 117 us,
// 0.58 PFLOP/s of products, bound by the loop over blocks (matrix units 30% busy, vector
// instructions 51%); 32 over 8192 (fp16) 28.7 us, bound by a part's start (5 us), its eight
// blocks (11), the store of its sums (3.5) and the join (6).
#pragma once

#include "kvattn_kernels.h"

namespace vbq {
namespace {

template <int G, int ROWS>
constexpr int kStages = G == 1 && ROWS <= 8 ? 4 : 2;

// Wavefronts a SIMD that registers are kept for.
template <int G, int SHARED_ROWS>
constexpr int kBothRoom = SHARED_ROWS == kRowTile ? (G >= 4 ? 1 : 2) : kRoomy<G, SHARED_ROWS> ? 4 : G * SHARED_ROWS > 64 ? 1 : 2;
// Shared tokens by the kernel for few rows (SHARED_ROWS up to 32), or for many (128).
template <int G, int SHARED_ROWS, bool FINE, int OWN_ROWS>
__global__ __launch_bounds__(256, (kBothRoom<G, SHARED_ROWS>)) void k_kv4_attn_both(KvAttn shared, KvAttn own, uint32_t shared_tiles, uint32_t shared_groups) {
  constexpr bool TILE = SHARED_ROWS == kRowTile;
  constexpr int FEW = TILE ? 4 : SHARED_ROWS;
  constexpr int A = TILE ? TileLds<G>::kRaw + TileLds<G>::kKeys + TileLds<G>::kVals
                         : few_rows_lds<G, FEW, kStages<G, FEW>, 4>();
  constexpr int B = few_rows_lds<G, OWN_ROWS, kStages<G, OWN_ROWS>, 4>();
  __shared__ __attribute__((aligned(16))) uint8_t lds[A > B ? A : B];
  constexpr int WML = FEW > OWN_ROWS ? FEW : OWN_ROWS;
  __shared__ float wml[4 * WML * 2];
  __shared__ uint32_t last;
  if (blockIdx.x < shared_groups) {
    if constexpr (TILE)
      tile_rows<G, FINE, kShared>(shared, lds, lds + TileLds<G>::kRaw, lds + TileLds<G>::kRaw + TileLds<G>::kKeys,
                                  blockIdx.x % shared_tiles, blockIdx.x / shared_tiles);
    else
      few_rows<G, FEW, kStages<G, FEW>, kShared, 4>(shared, lds, reinterpret_cast<float (*)[FEW][2]>(wml), &last,
                                                    blockIdx.x, shared_groups);
  } else {
    few_rows<G, OWN_ROWS, kStages<G, OWN_ROWS>, kOwn, 4>(own, lds, reinterpret_cast<float (*)[OWN_ROWS][2]>(wml), &last,
                                                         blockIdx.x - shared_groups, gridDim.x - shared_groups);
  }
}

// Joins a row's sums: of the parts of its group's shared tokens (TILE: as the kernel for
// many rows leaves them; else one part), and of its sequence's own. Where there are many
// parts, slices of a row's threads take every SLICESth, eight loads on their way at a
// time. blockIdx.x is the tile as in the kernel for many rows. Bound by reading the sums:
// 34 MB of 32 parts 8.4 us, 17 MB 6.0. Whole calls by one and by four slices, us: 32 parts of
// 8 tiles of heads of 128 31.5 and 28.6, 16 of 16 44.7 and 43.7, 10 of 48 76.5 and 76.8, 8 of 64
// 95.1 and 96.8, 4 of 128 119.6 and 125.8; 32 of heads of 64 24.2 and 20.8, of 256 59.7 and 55.2.
template <int G, bool TILE, int SLICES>
__global__ __launch_bounds__(256) void k_kv4_attn_meet(KvAttn a, const float* own, const float* own_ml) {
  constexpr int D = 64 * G, LANES = D / 4, ROWS = 256 / (LANES * SLICES), AT_ONCE = TILE ? 8 : 1;
  static_assert(ROWS >= 1, "a row fits a workgroup");
  __shared__ __attribute__((aligned(16))) f32x4 other[SLICES > 1 ? (SLICES - 1) * ROWS * LANES : 1];
  __shared__ f32x2 other_ml[SLICES > 1 ? (SLICES - 1) * ROWS : 1];
  const int c = (int)threadIdx.x % LANES, slot = (int)threadIdx.x / LANES, slice = slot / ROWS, in = slot % ROWS;
  const uint32_t bh_n = (uint32_t)(a.batch * a.cache.heads), bh = blockIdx.x % bh_n;
  const int g = (int)(bh / (uint32_t)a.cache.heads), head = (int)(bh % (uint32_t)a.cache.heads);
  Seq sq;
  if (!seq_at<kShared>(a, g, sq)) return;
  const int rows = sq.nq * a.ratio, rts = (rows + kRowTile - 1) / kRowTile;
  const int rt = TILE ? rts - 1 - (int)(blockIdx.x / bh_n) : 0;
  if (rt < 0) return;
  const int in_tile = (int)blockIdx.y * ROWS + in, r = rt * kRowTile + in_tile;
  const bool mine = slot < SLICES * ROWS && r < rows && in_tile < kRowTile;
  const int qi = r / a.ratio, hh = r - qi * a.ratio;
  const int64_t o = (int64_t)(sq.c0 + qi) * a.n_heads + head * a.ratio + hh;
  int parts = 1;
  if constexpr (TILE) {
    const int per = part_blocks(a, sq.re);
    parts = (sq.re.nw + per - 1) / per;
  }
  const int64_t place = TILE ? (int64_t)blockIdx.x * a.parts * kRowTile + in_tile : o;
  const float* const sums = (TILE ? a.acc : a.sums) + place * D + 4 * c;
  const float* const ml = (TILE ? a.ml : a.sums_ml) + 2 * place;
  constexpr int STEP = kRowTile;   // rows between parts
  float low = -kNoMax, sum = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](const f32x2& x, const f32x4& y) {
    const float to = fminf(low, x.x), f = __builtin_amdgcn_exp2f(to - low), h = __builtin_amdgcn_exp2f(to - x.x);
    sum = __builtin_fmaf(sum, f, x.y * h);
    v = v * f + y * h;
    low = to;
  };
  if (mine) {
    f32x2 x_own = {-kNoMax, 0.f};
    f32x4 y_own = {0.f, 0.f, 0.f, 0.f};
    if (slice == 0) {
      x_own = *reinterpret_cast<const f32x2*>(own_ml + 2 * o);
      y_own = *reinterpret_cast<const f32x4*>(own + o * D + 4 * c);
    }
    for (int p0 = slice; p0 < parts; p0 += SLICES * AT_ONCE) {
      f32x2 x[AT_ONCE];
      f32x4 y[AT_ONCE];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int p = p0 + i * SLICES;
        if (i && p >= parts) continue;
        x[i] = *reinterpret_cast<const f32x2*>(ml + (int64_t)p * (2 * STEP));
        y[i] = *reinterpret_cast<const f32x4*>(sums + (int64_t)p * (STEP * D));
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i)
        if (i == 0 || p0 + i * SLICES < parts) add(x[i], y[i]);
    }
    if (slice == 0) {
      if (x_own.y == kLeftOut) low = __builtin_nanf("");   // (no sum's base: the row is not written)
      else add(x_own, y_own);
    } else {
      other[((slice - 1) * ROWS + in) * LANES + c] = v;
      if (c == 0) other_ml[(slice - 1) * ROWS + in] = f32x2{low, sum};
    }
  }
  if constexpr (SLICES > 1) __syncthreads();
  if (!mine || slice || low != low) return;
#pragma unroll
  for (int i = 0; i < SLICES - 1; ++i) add(other_ml[i * ROWS + in], other[(i * ROWS + in) * LANES + c]);
  answer_row<D>(a, o, c, v, sum, low);
}

template <Part PART, int G>
void launch_few(const KvAttn& a, const KvAttnPlan& p, hipStream_t s) {
  const dim3 grid((uint32_t)p.grid);
#define VBQ_CALL(ROWS) k_kv4_attn<G, ROWS, kStages<G, ROWS>, PART><<<grid, (64 * kWaves<G, ROWS>), 0, s>>>(a)
  if (PART != kShared && p.rows == 4) { if constexpr (PART != kShared) VBQ_CALL(4); }   // (shared: 8 at least)
  else if (p.rows == 8) VBQ_CALL(8);
  else if (G == 4 || p.rows == 16) VBQ_CALL(16);
  else if constexpr (G < 4) VBQ_CALL(32);
#undef VBQ_CALL
}

template <int G, int OWN_ROWS>
void launch_both(const KvAttn& sh, const KvAttnPlan& sp, const KvAttn& own, const KvAttnPlan& op, hipStream_t s) {
  const bool tile = sp.rows == kRowTile;
  const uint32_t groups = (uint32_t)(sp.grid * (tile ? sh.parts : 1));
  const dim3 grid(groups + (uint32_t)op.grid);
#define VBQ_CALL(ROWS, FINE) k_kv4_attn_both<G, ROWS, FINE, OWN_ROWS><<<grid, 256, 0, s>>>(sh, own, (uint32_t)sp.grid, groups)
  if (tile) {
    if (sh.bf16) VBQ_CALL(kRowTile, false);
    else VBQ_CALL(kRowTile, true);
  } else if (G == 4 || sp.rows <= 16) {
    if (OWN_ROWS < 16 && sp.rows <= 8) { if constexpr (OWN_ROWS < 16) VBQ_CALL(8, false); }
    else VBQ_CALL(16, false);
  } else if constexpr (G < 4) {
    VBQ_CALL(32, false);
  }
#undef VBQ_CALL
}

template <int G>
hipError_t launch_shared(const KvAttn& sh, const KvAttnPlan& sp, const KvAttn& own, const KvAttnPlan& op, bool each,
                         hipStream_t s) {
  if (each) {
    launch_few<kEach, G>(own, op, s);
    return hipGetLastError();
  }
  const bool tile = sp.rows == kRowTile, any = sp.grid > 0 && sh.max_kv > 0;
  const bool together = !(G == 4 && tile && op.grid > 256);   // (both sides measured above)
  if (any && together && op.rows <= 16 && (tile || sp.rows >= op.rows)) {
    if (op.rows == 4) launch_both<G, 4>(sh, sp, own, op, s);
    else if (op.rows == 8) launch_both<G, 8>(sh, sp, own, op, s);
    else launch_both<G, 16>(sh, sp, own, op, s);
  } else {
    if (any && tile) {
      const dim3 tiles((uint32_t)sp.grid, (uint32_t)sh.parts);
      if (sh.bf16) k_kv4_attn_tile<G, false, kShared><<<tiles, 256, 0, s>>>(sh);
      else k_kv4_attn_tile<G, true, kShared><<<tiles, 256, 0, s>>>(sh);
    } else if (any) {
      launch_few<kShared, G>(sh, sp, s);
    }
    if (op.rows == kRowTile) {
      const dim3 tiles((uint32_t)op.grid, (uint32_t)own.parts);
      if (own.bf16) k_kv4_attn_tile<G, false, kOwn><<<tiles, 256, 0, s>>>(own);
      else k_kv4_attn_tile<G, true, kOwn><<<tiles, 256, 0, s>>>(own);
      if (own.parts > 1) k_kv4_attn_join<G, kOwn><<<dim3((uint32_t)op.grid, kRowTile * G / 16), 256, 0, s>>>(own);
    } else {
      launch_few<kOwn, G>(own, op, s);
    }
  }
  if (any) {
    constexpr int one = 256 / (16 * G), four = 256 / (64 * G);   // rows of a workgroup, by slices
    const dim3 by_one((uint32_t)(tile ? sp.grid : sp.tiles), (uint32_t)((sp.rows + one - 1) / one));
    if (!tile) k_kv4_attn_meet<G, false, 1><<<by_one, 256, 0, s>>>(sh, own.sums, own.sums_ml);
    else if (sh.parts <= 8) k_kv4_attn_meet<G, true, 1><<<by_one, 256, 0, s>>>(sh, own.sums, own.sums_ml);
    else k_kv4_attn_meet<G, true, 4><<<dim3((uint32_t)sp.grid, kRowTile / four), 256, 0, s>>>(sh, own.sums, own.sums_ml);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace vbq
