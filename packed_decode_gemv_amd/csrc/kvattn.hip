// Sizes and launches of attention over the 4-bit key/value cache; the kernels are in
// kvattn_kernels.h.
#include "kvattn_kernels.h"

namespace vbq {

// Rows a tile takes: columns of one MFMA tile, or two tiles; above 32 the tile
// kernel, and above 16 for heads of 256, where two column tiles do not fit the
// registers (8 sequences x 20 rows x 4 heads, 20206 tokens: 46 against 64 us; heads
// of 192: 39 against 34). Short tiles are not cut (a workgroup each, and no parts to work out
// and join): up to five blocks a wavefront, or twelve where the tiles alone fill
// the chip. Uncut and cut, heads of 128, 4 rows: 8 tiles of 19 blocks 9.4 and
// 10.0 us, of 29 blocks 12.0 and 10.1; 256 tiles of 38 blocks 16.4 and 18.0,
// of 63 blocks 21.8 and 22.2.
KvAttnPlan kv4_attn_plan(int batch, int heads, int ratio, int groups, int total_q, int max_q, int max_kv, int window,
                         int sinks) {
  KvAttnPlan p;
  p.threads = 256;
  const int64_t rows = (int64_t)max_q * ratio;
  int64_t blocks = ((int64_t)max_kv + kKvBlock - 1) / kKvBlock;
  if (window) {   // (a tile's rows: at most 128 queries)
    const int64_t most = ((int64_t)sinks + window + (max_q < kRowTile ? max_q : kRowTile)) / kKvBlock + 3;
    blocks = blocks < most ? blocks : most;
  }
  if (rows > (groups == 4 ? 16 : 32)) {   // many rows: the tile kernel
    p.rows = kRowTile;
    p.tiles = (int64_t)batch * heads * ((rows + p.rows - 1) / p.rows);
    // Where tiles leave places on the chip (two workgroups a CU, one with large heads), parts fill them.
    const int64_t fill = (groups <= 3 ? 512 : 256) / (p.tiles ? p.tiles : 1), most = blocks / kLeastTilePart;
    const int64_t parts = fill < most ? fill : most;
    p.parts = (int32_t)(parts < 1 ? 1 : parts < kTileParts ? parts : kTileParts);
    p.places = p.parts > 1 ? p.tiles * p.parts : 0;
    // (no sequence has more queries than the call: a workgroup beyond them would find no tile)
    const int64_t most_rows = (int64_t)(max_q < total_q ? max_q : total_q) * ratio;
    p.grid = (int64_t)batch * heads * ((most_rows + p.rows - 1) / p.rows);
    return p;
  }
  p.rows = rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  p.tiles = (int64_t)batch * heads;
  // Tiles longer than total / parts are cut, so there are at most `parts` parts
  // beyond one a tile, and on average half a part a tile: the aim leaves room
  // for those where one workgroup of eight wavefronts or two of four fit a CU, so
  // that all run at once (a second round: 34 against 23 us for 128 tiles of 16 rows).
  const bool cut = p.tiles <= VBQ_KV4_COUNTERS && blocks > (p.tiles < 256 ? 5 : 12) * 4 &&
                   p.tiles * blocks < INT32_MAX - 65536;
  const int fill = groups <= 2 && p.rows >= 16 ? kParts / 2 : kParts;   // (eight wavefronts each)
  const int spare = groups <= 2 && p.rows <= 8 ? 0 : (int)(p.tiles < fill ? p.tiles : fill) / 2;
  p.parts = cut ? fill - spare : 0;
  p.grid = cut ? p.parts + p.tiles : p.tiles;
  p.places = cut ? p.grid : 0;
  p.threads = 64 * few_row_waves(groups, p.rows);
  return p;
}

hipError_t launch_kv4_attention(const KvAttn& a, const KvAttnPlan& p, hipStream_t s) {
  const dim3 grid((uint32_t)p.grid);
#define VBQ_CALL(G, ROWS, ST) k_kv4_attn<G, ROWS, ST><<<grid, (64 * kWaves<G, ROWS>), 0, s>>>(a)
#define VBQ_CALL2(G, FEW, ST)                \
  if (p.rows == 4) VBQ_CALL(G, 4, FEW);      \
  else if (p.rows == 8) VBQ_CALL(G, 8, FEW); \
  else VBQ_CALL(G, 16, ST)
#define VBQ_CALL3(G, FEW, ST)                  \
  if (p.rows == 32) VBQ_CALL(G, 32, ST);       \
  else VBQ_CALL2(G, FEW, ST)
#define VBQ_TILE(G)                                               \
  if (a.bf16) k_kv4_attn_tile<G, false><<<tiles, 256, 0, s>>>(a); \
  else k_kv4_attn_tile<G, true><<<tiles, 256, 0, s>>>(a);         \
  if (a.parts > 1) k_kv4_attn_join<G><<<dim3((uint32_t)p.grid, kRowTile * G / 16), 256, 0, s>>>(a)
  if (p.rows == kRowTile) {
    const dim3 tiles((uint32_t)p.grid, (uint32_t)a.parts);
    switch (a.cache.groups) {
      case 1: VBQ_TILE(1); break;
      case 2: VBQ_TILE(2); break;
      case 3: VBQ_TILE(3); break;
      default: VBQ_TILE(4); break;
    }
    return hipGetLastError();
  }
  switch (a.cache.groups) {
    case 1: VBQ_CALL3(1, 4, 2); break;
    case 2: VBQ_CALL3(2, 2, 2); break;
    case 3: VBQ_CALL3(3, 2, 2); break;
    default: VBQ_CALL2(4, 2, 2); break;
  }
#undef VBQ_CALL3
#undef VBQ_CALL2
#undef VBQ_CALL
#undef VBQ_TILE
  return hipGetLastError();
}

}  // namespace vbq
