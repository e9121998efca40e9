// Attention of sequences that have their first tokens in common (meaning in vbq.h):
// the kernels of kvattn_kernels.h in two launches, one over the groups' shared tokens,
// where the rows of all of a group's sequences make the tiles, and one over the
// sequences' own tokens, which joins its sums with those of the first.
#include "kvattn_kernels.h"

namespace vbq {

template <Part PART>
static void launch_part(const KvAttn& a, const KvAttnPlan& p, hipStream_t s) {
  const dim3 grid((uint32_t)p.grid);
#define VBQ_CALL(G, ROWS, ST) k_kv4_attn<G, ROWS, ST, PART><<<grid, (64 * kWaves<G, ROWS>), 0, s>>>(a)
#define VBQ_CALL2(G, FEW, ST)                \
  if (p.rows == 4) VBQ_CALL(G, 4, FEW);      \
  else if (p.rows == 8) VBQ_CALL(G, 8, FEW); \
  else VBQ_CALL(G, 16, ST)
#define VBQ_CALL3(G, FEW, ST)                  \
  if (p.rows == 32) VBQ_CALL(G, 32, ST);       \
  else VBQ_CALL2(G, FEW, ST)
#define VBQ_TILE(G)                                                     \
  if (a.bf16) k_kv4_attn_tile<G, false, PART><<<tiles, 256, 0, s>>>(a); \
  else k_kv4_attn_tile<G, true, PART><<<tiles, 256, 0, s>>>(a);         \
  if (a.parts > 1) k_kv4_attn_join<G, PART><<<dim3((uint32_t)p.grid, kRowTile * G / 16), 256, 0, s>>>(a)
  if (p.rows == kRowTile) {
    const dim3 tiles((uint32_t)p.grid, (uint32_t)a.parts);
    switch (a.cache.groups) {
      case 1: VBQ_TILE(1); break;
      case 2: VBQ_TILE(2); break;
      case 3: VBQ_TILE(3); break;
      default: VBQ_TILE(4); break;
    }
    return;
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
}

hipError_t launch_kv4_attention_shared(const KvAttn& shared, const KvAttnPlan& sp, const KvAttn& own,
                                       const KvAttnPlan& op, hipStream_t s) {
  if (sp.grid > 0 && shared.max_kv > 0) launch_part<kShared>(shared, sp, s);
  launch_part<kOwn>(own, op, s);
  return hipGetLastError();
}

}  // namespace vbq
