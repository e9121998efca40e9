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
constexpr int kMaxPieces = 512;

// Exchanges with the lanes 16 and 32 apart (the lane quarters of a column).
typedef uint32_t pair_t __attribute__((ext_vector_type(2)));
__device__ inline float rows_max(float v) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  pair_t p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  uint32_t x = p.x, y = p.y;
  v = fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
  u = __builtin_bit_cast(uint32_t, v);
  p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  x = p.x, y = p.y;
  return fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ inline float rows_sum(float v) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  pair_t p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  uint32_t x = p.x, y = p.y;
  v = __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
  u = __builtin_bit_cast(uint32_t, v);
  p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  x = p.x, y = p.y;
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
// Inclusive sum over the lanes of a wavefront.
__device__ inline int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
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

// A block's copy to LDS: 16 bytes a lane and instruction, no registers, so
// later blocks are on their way while one is worked on.
template <int G>
constexpr int kCopies = (kKvGroupBytes * G + 1023) / 1024;
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

// A sequence of the call as the kernels see it.
struct Seq {
  int32_t c0, nq, len, first;   // first row of q, queries, tokens held, position of query 0
  Reach re;
  int32_t blocks, tiles;        // blocks of every tile, and tiles: heads * row tiles
};
// False (and nothing to do) for numbers that do not fit.
__device__ inline bool seq_from(const KvAttn& a, int rows_per_tile, int c0, int c1, int len, Seq& s) {
  const int64_t nq = (int64_t)c1 - c0;
  s.blocks = s.tiles = 0;
  if (c0 < 0 || nq < 0 || c1 > a.total_q || nq > a.max_q || len < 0 || len > a.max_kv ||
      (int64_t)len > ((int64_t)a.width << (a.cache.block_shift + 5)))
    return false;
  s.c0 = c0;
  s.nq = (int32_t)nq;
  s.len = len;
  s.first = len - s.nq;
  if (nq == 0) return true;
  s.re = reach(len, a.causal ? s.first : len - 1, len - 1, a.window, a.sinks);
  s.blocks = s.re.ns + s.re.nw;
  s.tiles = a.cache.heads * ((s.nq * a.ratio + rows_per_tile - 1) / rows_per_tile);
  return true;
}

// The token axes of all tiles laid end to end: sequence by sequence, tile by
// tile, block by block. It is cut into equal pieces of `chunk` blocks, one a
// workgroup, so the work is even whatever the lengths are; a tile that a cut
// crosses leaves partial sums.
struct Line {
  int32_t total, chunk;
  // lane l: sequence base + l of the batch, and the line's units up to its end
  int32_t base, c0, c1, len, incl;
};
__device__ inline void line_load(const KvAttn& a, int rows_per_tile, uint32_t lane, int base, int before, bool report,
                                 Line& l) {
  const int b = base + (int)lane;
  l.base = base;
  l.c0 = l.c1 = l.len = 0;
  int units = 0;
  if (b < a.batch) {
    l.c0 = a.cu[b];
    l.c1 = a.cu[b + 1];
    l.len = a.lens[b];
    Seq s;
    if (seq_from(a, rows_per_tile, l.c0, l.c1, l.len, s)) units = s.blocks * s.tiles;
    else if (report) kv_flag(a.cache, VBQ_KV4_FLAG_LENGTH);
  }
  l.incl = before + wave_scan(units);
}
__device__ inline void line_of(const KvAttn& a, int rows_per_tile, uint32_t lane, bool report, Line& l) {
  l.total = 0;
  for (int base = 0; base < a.batch; base += 64) {
    line_load(a, rows_per_tile, lane, base, l.total, report, l);
    l.total = __builtin_amdgcn_readlane(l.incl, 63);
  }
  const uint32_t c = ((uint32_t)l.total + (uint32_t)a.pieces - 1u) / (uint32_t)a.pieces;
  l.chunk = max((int)c, a.min_chunk);
}
// The sequence that unit `pos` (less than the total) belongs to.
__device__ inline int line_find(const KvAttn& a, int rows_per_tile, uint32_t lane, int pos, Line& l) {
  if (a.batch > 64) {
    int before = 0;
    for (int base = 0;; base += 64) {
      line_load(a, rows_per_tile, lane, base, before, false, l);
      before = __builtin_amdgcn_readlane(l.incl, 63);
      if (before > pos || base + 64 >= a.batch) break;
    }
  }
  const uint64_t past = __ballot(l.incl > pos);
  return l.base + (past ? __builtin_ctzll(past) : 63);
}
__device__ inline int line_before(const Line& l, int lane_of_seq, int first) {   // units before a sequence
  return lane_of_seq ? __builtin_amdgcn_readlane(l.incl, lane_of_seq - 1) : first;
}

// Where a piece's partial sums of a tile lie: the tile that a piece starts in
// the middle of is its slot 0, one that it starts and does not end its slot 1.
template <int G, int NT>
struct Slot {
  float *acc, *ml;
  __device__ Slot(const KvAttn& a, int piece, bool starts) {
    const int64_t n = 2 * piece + (starts ? 1 : 0);
    acc = a.acc + n * (16 * NT) * (64 * G);
    ml = a.ml + n * (16 * NT) * 2;
  }
};

// STAGES blocks a wavefront in LDS, STAGES - 1 of them on their way.
template <int G, int NT, int STAGES>
__global__ __launch_bounds__(64 * kWaves, G * NT > 4 ? 1 : 2) void k_kv4_attn(KvAttn a) {
  constexpr int D = 64 * G, ROWS = 16 * NT, PITCH = D + 4, BYTES = kKvGroupBytes * G;
  constexpr int RING = kWaves * STAGES * BYTES, SUMS = kWaves * 16 * PITCH * 4;
  __shared__ __attribute__((aligned(16))) uint8_t ring[RING > SUMS ? RING : SUMS];
  __shared__ float wml[kWaves][ROWS][2];
  float* const buf = reinterpret_cast<float*>(ring);   // the wavefronts' sums, after a tile
  const uint32_t tid = threadIdx.x, lane = tid & 63u, col = lane & 15u, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t* const own_ring = ring + wave * STAGES * BYTES;
  const uint32_t ring_lds = lds_addr(own_ring);
  const Decode dc;

  // This workgroup's piece of the line, or its tile.
  int pos = 0, end = 1, b;
  Line line;
  if (a.pieces) {
    line_of(a, ROWS, lane, blockIdx.x == 0 && wave == 0, line);
    pos = (int)min((int64_t)blockIdx.x * line.chunk, (int64_t)line.total);
    end = (int)min((int64_t)pos + line.chunk, (int64_t)line.total);
    if (pos >= end) return;
    b = line_find(a, ROWS, lane, pos, line);
  } else {
    b = (int)(blockIdx.x / (uint32_t)(a.cache.heads * a.row_tiles));
  }
  for (bool fresh = true; pos < end; fresh = false) {
  Seq sq;
  int tile, i0, i1;
  if (a.pieces) {
    const int at = b - line.base;   // below 64: every sequence but the last ends inside the lanes' ones
    const int past = __builtin_amdgcn_readlane(line.incl, at);
    if (past <= pos) {   // on to the next sequence
      if (++b >= a.batch) return;
      if (at == 63) line_load(a, ROWS, lane, b, past, false, line);
      continue;
    }
    seq_from(a, ROWS, __builtin_amdgcn_readlane(line.c0, at), __builtin_amdgcn_readlane(line.c1, at),
             __builtin_amdgcn_readlane(line.len, at), sq);
    const uint32_t rel = (uint32_t)(pos - (past - sq.blocks * sq.tiles));
    tile = (int)(rel / (uint32_t)sq.blocks);
    i0 = (int)rel - tile * sq.blocks;
    i1 = min(sq.blocks, i0 + (end - pos));
    pos += i1 - i0;
  } else {
    if (!seq_from(a, ROWS, a.cu[b], a.cu[b + 1], a.lens[b], sq)) {
      if (tid == 0) kv_flag(a.cache, VBQ_KV4_FLAG_LENGTH);
      return;
    }
    tile = (int)(blockIdx.x % (uint32_t)(a.cache.heads * a.row_tiles));
    if (tile >= sq.tiles) return;
    i0 = 0;
    i1 = sq.blocks;
    pos = end;
  }
  const Reach re = sq.re;
  const int c0 = sq.c0, len = sq.len, first = sq.first, rows = sq.nq * a.ratio;
  const int rts = (rows + ROWS - 1) / ROWS;
  const int head = tile / rts, r0 = (tile - head * rts) * ROWS, r1 = min(rows, r0 + ROWS);
  const int p_min = a.causal ? first + r0 / a.ratio : len - 1;
  const int p_max = a.causal ? first + (r1 - 1) / a.ratio : len - 1;
  if (!fresh) __syncthreads();   // the ring held the last tile's sums

  // Queries, on their way while the first pages are looked up.
  u32x4 qraw[NT][G][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 16 * nt + (int)col;
    const int qi = r / a.ratio, hh = r - qi * a.ratio;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        qraw[nt][g][st] = u32x4{0, 0, 0, 0};
        if (r < rows)
          qraw[nt][g][st] = *reinterpret_cast<const u32x4*>(a.q + (int64_t)(c0 + qi) * a.q_ts +
                                                            (int64_t)(head * a.ratio + hh) * a.q_hs + 64 * g +
                                                            32 * st + 8 * quarter);
      }
  }

  // The wavefront's blocks: copies run STAGES - 1 ahead.
  const uint32_t in_page = (1u << a.cache.block_shift) - 1u;
  int pages = -1;   // lane i: the page of the wavefront's block i (of 64 at a time)
  uint64_t gone = 0, gone_before = 0;   // those that are not in the cache, and of the 64 before
  auto block_of = [&](int idx) { return idx < re.ns ? idx : idx - re.ns + re.w0; };
  auto start_copy = [&](int it) {
    const int idx = i0 + wave + kWaves * it;
    if ((it & 63) == 0) {
      const int next = idx + kWaves * (int)lane;
      pages = 0;
      bool bad = false;
      if (next < i1) {
        pages = a.table[(int64_t)b * a.width + (block_of(next) >> a.cache.block_shift)];
        bad = (uint32_t)pages >= (uint32_t)a.cache.n_pages;
      }
      if (bad) {
        pages = 0;   // copied, and left out of the sums
        kv_flag(a.cache, VBQ_KV4_FLAG_PAGE);
      }
      gone_before = gone;
      gone = __ballot(bad);
    }
    const int page = __builtin_amdgcn_readlane(pages, it & 63);
    copy_block<G>(ring_lds + (uint32_t)(it % STAGES) * BYTES,
                  kv_block(a.cache, G, (uint32_t)page, head, (uint32_t)block_of(idx) & in_page), lane);
  };
  const int count = i0 + wave < i1 ? (i1 - i0 - wave + kWaves - 1) / kWaves : 0;
#pragma unroll
  for (int it = 0; it < STAGES - 1; ++it)
    if (it < count) start_copy(it);

  // Queries: B operands per group and 32-channel step, their sums per group,
  // and what each lane's column sees.
  half8_t qf[NT][G][2];
  float qsum[NT][G], to_log2[NT];
  int hi[NT], lo[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 16 * nt + (int)col;
    const bool in = r < rows;
    const int qi = r / a.ratio;
    float x[G][2][8];
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const u32x4 w = qraw[nt][g][st];
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

  for (int it = 0; it < count; ++it) {
    // This block's copy has landed (later ones may be on their way), and the
    // reads of the buffer that the next copy takes are done.
    if (it + STAGES - 1 <= count)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kCopies<G> * (STAGES - 2)) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    const int ahead = it + STAGES - 1;
    if (ahead < count) start_copy(ahead);
    // (the pages of the 64 blocks after may have been looked up already)
    if ((((it ^ min(ahead, count - 1)) >> 6 ? gone_before : gone) >> (it & 63)) & 1u) continue;
    const int blk = block_of(i0 + wave + kWaves * it);
    const uint8_t* const k = own_ring + (it % STAGES) * BYTES;

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
  const bool whole = i0 == 0 && i1 == sq.blocks;
  const Slot<G, NT> slot(a, blockIdx.x, i0 == 0);
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
        *reinterpret_cast<f32x4*>(slot.acc + rr * D + 4 * c) = v;
        if (c == 0) *reinterpret_cast<f32x2*>(slot.ml + 2 * rr) = f32x2{top, sum};
      }
    }
  }
  }
}

// Joins the partial sums of tiles that the line's cuts cross, piece by piece in
// order, and answers tiles that see no block at all. One workgroup a tile.
constexpr int kJoinThreads = 512;
template <int G, int NT>
__global__ __launch_bounds__(kJoinThreads) void k_kv4_join(KvAttn a) {
  constexpr int D = 64 * G, ROWS = 16 * NT, ROW_LANES = kJoinThreads / 16;
  __shared__ float factor[16][kMaxPieces];
  __shared__ f32x4 share[kJoinThreads];
  __shared__ float total[16][2];
  const uint32_t tid = threadIdx.x, lane = tid & 63u;
  const uint32_t per = (uint32_t)(a.cache.heads * a.row_tiles);
  const int b = (int)(blockIdx.x / per), tile = (int)(blockIdx.x % per);
  Seq sq;
  if (!seq_from(a, ROWS, a.cu[b], a.cu[b + 1], a.lens[b], sq) || tile >= sq.tiles) return;
  const int rows = sq.nq * a.ratio, rts = (rows + ROWS - 1) / ROWS;
  const int head = tile / rts, r0 = (tile - head * rts) * ROWS;
  int p0 = 0, pieces = 0;
  if (sq.blocks > 0) {
    Line line;
    line_of(a, ROWS, lane, false, line);
    int before = 0;
    if (a.batch > 64)
      for (int base = 0;; base += 64) {   // the lanes' sequences are to hold b
        line_load(a, ROWS, lane, base, before, false, line);
        if (b < base + 64) break;
        before = __builtin_amdgcn_readlane(line.incl, 63);
      }
    const uint32_t u = (uint32_t)(line_before(line, b - line.base, before) + tile * sq.blocks);
    p0 = (int)(u / (uint32_t)line.chunk);
    pieces = (int)((u + (uint32_t)sq.blocks - 1u) / (uint32_t)line.chunk) - p0 + 1;
    if (pieces == 1) return;   // whole: its workgroup has answered
  }
#pragma unroll 1
  for (int nt = 0; nt < NT; ++nt) {
    const int nrow = min(16, rows - r0 - 16 * nt);
    if (nrow <= 0) break;
    __syncthreads();
    {   // 32 lanes a row: the common maximum, each piece's factor, the sum
      const int row = (int)tid / ROW_LANES, j = (int)tid % ROW_LANES;
      float top = kNoMax, sum = 0.f;
      if (row < nrow) {
        for (int p = j; p < pieces; p += ROW_LANES) {
          const float m = Slot<G, NT>(a, p0 + p, p == 0).ml[2 * (16 * nt + row)];
          factor[row][p] = m;
          top = fmaxf(top, m);
        }
      }
#pragma unroll
      for (int d = 1; d < ROW_LANES; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
      if (row < nrow) {
        for (int p = j; p < pieces; p += ROW_LANES) {
          const float f = __builtin_amdgcn_exp2f(factor[row][p] - top);
          factor[row][p] = f;
          sum += f * Slot<G, NT>(a, p0 + p, p == 0).ml[2 * (16 * nt + row) + 1];
        }
      }
#pragma unroll
      for (int d = 1; d < ROW_LANES; d <<= 1) sum += __shfl_xor(sum, d, 64);
      if (j == 0) {
        total[row][0] = top;
        total[row][1] = sum;
      }
    }
    __syncthreads();
    // Threads beyond the rows' outputs share the pieces.
    const int ne = nrow * (D / 4), parts = ne <= kJoinThreads / 2 ? kJoinThreads / ne : 1;
    for (int e0 = 0; e0 < ne; e0 += kJoinThreads) {
      const int e = parts > 1 ? (int)tid % ne : e0 + (int)tid, part = parts > 1 ? (int)tid / ne : 0;
      const int row = e / (D / 4), c = e % (D / 4);
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      if (e < ne && part < parts) {
#pragma unroll 4
        for (int p = part; p < pieces; p += parts)
          v += *reinterpret_cast<const f32x4*>(Slot<G, NT>(a, p0 + p, p == 0).acc + (16 * nt + row) * D + 4 * c) *
               factor[row][p];
      }
      if (parts > 1) {
        share[tid] = v;
        __syncthreads();
        if (part == 0)
          for (int i = 1; i < parts; ++i) v += share[e + i * ne];
      }
      if (e < ne && part == 0) {
        const int r = r0 + 16 * nt + row, qi = r / a.ratio, hh = r - qi * a.ratio;
        const int64_t o = (int64_t)(sq.c0 + qi) * a.n_heads + head * a.ratio + hh;
        const float top = total[row][0], sum = total[row][1];
        const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
        store4(a, o * D + 4 * c, v * inv);
        if (a.lse && c == 0) a.lse[o] = (top + __builtin_amdgcn_logf(sum) - kProbShift) * kLn2;
      }
    }
  }
}

}  // namespace

// Rows a tile takes: one column tile of the MFMA, or two. Pieces of the line:
// two workgroups a CU. A tile is not cut (a workgroup each, no join) when there
// are enough of them to fill the chip or the tiles are short.
KvAttnPlan kv4_attn_plan(int batch, int heads, int ratio, int groups, int max_q, int max_kv, int window, int sinks) {
  KvAttnPlan p;
  const int64_t rows = (int64_t)max_q * ratio;
  p.rows = rows <= 16 ? 16 : 32;
  p.row_tiles = rows > 0 ? (int32_t)((rows + p.rows - 1) / p.rows) : 1;
  p.tiles = (int64_t)batch * heads * p.row_tiles;
  int64_t blocks = ((int64_t)max_kv + kKvBlock - 1) / kKvBlock;
  if (window) {
    const int64_t most = ((int64_t)sinks + window + max_q) / kKvBlock + 3;
    blocks = blocks < most ? blocks : most;
  }
  p.pieces = p.tiles < 2048 && blocks > 4 * kWaves && p.tiles * blocks < INT32_MAX - 65536 ? kMaxPieces : 0;
  return p;
}

hipError_t launch_kv4_attention(const KvAttn& a, const KvAttnPlan& p, int batch, hipStream_t s) {
  if (p.tiles > INT32_MAX) return hipErrorNotSupported;
  const dim3 grid(p.pieces ? (uint32_t)p.pieces : (uint32_t)p.tiles);
#define VBQ_CALL(G, NT, ST)                                                           \
  do {                                                                                \
    k_kv4_attn<G, NT, ST><<<grid, 64 * kWaves, 0, s>>>(a);                            \
    if (p.pieces) k_kv4_join<G, NT><<<(uint32_t)p.tiles, kJoinThreads, 0, s>>>(a);    \
  } while (0)
#define VBQ_CALL2(G, ST)                      \
  if (p.rows == 16) VBQ_CALL(G, 1, ST);       \
  else VBQ_CALL(G, 2, ST)
  switch (a.cache.groups) {
    case 1: VBQ_CALL2(1, 4); break;
    case 2: VBQ_CALL2(2, 4); break;
    case 3: VBQ_CALL2(3, 2); break;
    default: VBQ_CALL2(4, 2); break;
  }
#undef VBQ_CALL2
#undef VBQ_CALL
  return hipGetLastError();
}

}  // namespace vbq
