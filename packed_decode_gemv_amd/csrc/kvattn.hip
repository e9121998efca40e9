// Attention over the 4-bit key/value cache (layout and meaning in vbq.h).
//
// Rows are the (query token, query head) pairs that share a key/value head:
// row r of a sequence is query r / ratio, head r % ratio of the group. Up to 32
// rows a sequence and head (16 for heads of 256) take k_kv4_attn, more take
// k_kv4_attn_tile (below).
//
// k_kv4_attn: a workgroup of four or eight wavefronts takes a tile (all rows of
// one sequence and head), or a part of its token axis; wavefront w takes every
// fourth (eighth) block of 32 tokens and keeps its own running maximum, sum and
// output in registers. The wavefronts are joined in LDS, the parts in the
// workspace by the last workgroup that finishes.
//
// Scores. S^T = K Q^T by 16x16x32 fp16 MFMAs: A is a block's key codes, 16
// tokens by 32 channels of one group, B the queries. A code word holds eight
// channels of a token; a pair of codes masked out at bits 4-7 of each half is a
// pair of fp16 numbers c 2^-20. The group's scale and offset enter in
// fp32: score = sum_g s_g (codes . q)_g + o_g sum_g(q).
//   Where a code lies in the number matters, exact as it is anywhere. The
// matrix unit adds the eight products of a lane and cuts off what lies 24 bits
// below the largest, counted from its exponent; a subnormal has the exponent of
// 2^-14, so each zero in front of its bits costs one. At bits 4-7 it keeps a
// product of a code and a query down to 2^-18 of the largest query, at bits 0-3
// (c 2^-24, two shifts a word less) only to 2^-14: outputs of 32 sequences of
// 167000 tokens were off by 2.42e-4 (relative, whole tensor) with those and are
// off by 2.09e-4 with these, which is the rounding of the output itself. Normal
// numbers (c 2^-10, a product a pair) change nothing more there and take 55 us
// where these take 52 (and bits 0-3 took 51).
// Queries are scaled to a largest magnitude in [2^13, 2^14) per row (a power
// of two, undone in the score), so that fp16 holds them exactly down to 2^-30
// (bf16; 2^-27 fp16) of the row's largest.
//
// Output. O^T = V^T P^T by the same MFMA: A is the value codes, 16 channels by
// 32 tokens, again as c 2^-20; B the probabilities as they come out of
// the score MFMA: its result holds tokens 4 q + i of a column (row of the
// problem) in lane quarter q, and the cache orders a block's tokens so that
// those of both 16-token halves are the octet 8 q .. 8 q + 7, a value word. B
// carries p s (the token's scale in its group) as the sum of two fp16 numbers,
// so nothing is lost to fp16 but what lies 2^-37 below the largest; offsets
// enter as fp32 sums of p o per row and group. A wavefront holds p s times
// 2^S, S from the largest scale it has met.
//
// Few rows. With up to 8 (4) rows the MFMA's other columns hold copies of the
// queries, so every lane has every score of its row: lane part 0 .. 1 (0 .. 3)
// takes the scores of a half (quarter) of its octet's tokens, and scale,
// softmax and split are done once per score, not two (four) times.
//
// Bounds, heads of 128. 4 rows, 32 sequences of 167000 tokens in all, 8 heads:
// 193 MB in 51 us (3.8 TB/s; a plain read reaches 6.4). By clock stamps 4.5 us pass
// until the first block is there (arguments, lengths, table, block: each waits
// for the one before) and 2 and 3 us in the joins in LDS and in the workspace;
// with the launch that leaves about 39 us, 5.0 TB/s, for the blocks. One
// sequence of 131072 tokens: 151 MB in 42 us, 64 parts a tile to join.
// 16 heads of 16 sequences under a window of 1024: 38 MB in 15 us, the chain of
// dependent look-ups. 20 rows, 8 sequences of 20000 tokens in all, 8 heads: 24 MB
// in 25 us; three blocks a wavefront, of about 1.8 us each where one has a SIMD to
// itself (vector instructions and their latency), 4.6 us before the first, 7 us
// for the joins.
#include "kv4.h"

namespace vbq {
namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Wavefronts of a workgroup. Where registers allow two a SIMD but no more, eight
// that share one join do better than two workgroups of four (8 heads of 128 over
// 60000 tokens, 12 rows: 32 against 42 us; over 90000, 32 rows: 64 against 82; 64
// tiles of 20 rows of 80 blocks: 25 against 26).
constexpr int few_row_waves(int groups, int rows) { return groups <= 2 && rows >= 16 ? 8 : 4; }
template <int G, int ROWS>
constexpr int kWaves = few_row_waves(G, ROWS);
constexpr float kNoMax = -3e38f;     // running maximum before any token
// Probabilities are 2^(score * to_log2 - m) in one fma. m is a rounded product,
// so beyond 2^22 the exact product may pass it by more than a quarter, and
// beyond 2^31 by more than exp2 holds. Where a running maximum lies so far out,
// products are rounded first and m subtracted from them.
constexpr float kFar = 0x1p22f;
__device__ inline bool is_far(float m) { return m != kNoMax && fabsf(m) > kFar; }
__device__ inline float below(float score, float to_log2, float m) {
  float t = score * to_log2;
  asm("" : "+v"(t));   // (not one fma)
  return t - m;
}
constexpr int kParts = 512;          // workgroups that a launch aims at, at most
// Blocks of a part, at least. With 32 rows a part's sums are eight times those of
// 4 rows to join, and longer parts do no better even so (us with at least 8, 16,
// 24 and 32 blocks; heads of 128 but for the last): 64 tiles of 20 rows over 32
// blocks 19.5, 20.5, 20.5, 22.9; over 80 blocks 25.3, 25.3, 25.3, 27.8; over 125
// blocks 29.4, 29.2, 29.6, 29.1; 32 tiles of 24 rows over 94 blocks 21.4, 22.4, 24.1,
// 26.8; 16 tiles of 32 rows over 188 blocks 27.3, 25.8, 26.4, 28.0; 8 tiles over 625
// blocks 34.9, 34.8, 34.9, 34.4; 6 tiles of heads of 192 over 282 blocks 37.0, 37.1,
// 39.3, 43.5.
constexpr int kLeastPart = 8;

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
// Lane l of a row of 16 gets lane l + N's value (any value past the row's end);
// rotated by N.
template <int N>
__device__ inline uint32_t row_down(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x100 + N, 0xF, 0xF, true);
}
template <int N>
__device__ inline float row_turn(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xF, 0xF, true));
}
// Over the lanes that share a row of the problem: PARTS of a column's copies,
// then the lane quarters.
template <int PARTS>
__device__ inline float lanes_max(float v) {
  if constexpr (PARTS >= 2) v = fmaxf(v, row_turn<8>(v));
  if constexpr (PARTS == 4) v = fmaxf(v, row_turn<4>(v));
  return rows_max(v);
}
template <int PARTS>
__device__ inline float lanes_sum(float v) {
  if constexpr (PARTS >= 2) v += row_turn<8>(v);
  if constexpr (PARTS == 4) v += row_turn<4>(v);
  return rows_sum(v);
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

// Eight codes of a word as fp16 numbers c 2^-kCodeExp (subnormal), pairs (n, n + 4).
__device__ inline half8_t codes_of(uint32_t w) {
  u32x4 r;
  r.x = (w << 4) & 0x00F000F0u;
  r.y = w & 0x00F000F0u;
  r.z = (w >> 4) & 0x00F000F0u;
  r.w = (w >> 8) & 0x00F000F0u;
  return __builtin_bit_cast(half8_t, r);
}
constexpr int kCodeExp = 20;

__device__ inline half2_t pair_of(uint32_t w) { return __builtin_bit_cast(half2_t, w); }

// What brings a row's products, held times 2^-exp, to base two. Not 0, with which
// a hidden token's minus infinity would be NaN: at 2^-126 scores are below 2^-90.
__device__ inline float row_scale(const KvAttn& a, int exp) { return fmaxf(ldexpf(a.scale_log2, exp), 0x1p-126f); }

// N fp16 numbers from LDS.
template <int N>
struct Halves {
  uint32_t w[N > 1 ? N / 2 : 1];
  __device__ explicit Halves(const uint8_t* p) {
    if constexpr (N == 1) w[0] = *reinterpret_cast<const uint16_t*>(p);
    else if constexpr (N == 2) w[0] = *reinterpret_cast<const uint32_t*>(p);
    else if constexpr (N == 4) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      const u32x4 v = *reinterpret_cast<const u32x4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
  __device__ float operator[](int i) const {
    return (float)(i & 1 ? pair_of(w[i >> 1]).y : pair_of(w[i >> 1]).x);
  }
};

// A block's copy to LDS: 16 bytes a lane and instruction, no registers, so
// later blocks are on their way while one is worked on.
template <int G>
constexpr int kCopies = (kKvGroupBytes * G + 1023) / 1024;
// The address that lane i holds.
__device__ inline const uint8_t* lane_address(uint64_t v, int i) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, i);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), i);
  return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}
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
    const int lo = max(p_min, 0) - window + 1;   // first token in the window of any row that sees one
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
  uint32_t lo, hi;
  if (a.bf16) {
    typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
    const bf2_t x = {(__bf16)v[0], (__bf16)v[1]}, y = {(__bf16)v[2], (__bf16)v[3]};
    lo = __builtin_bit_cast(uint32_t, x);
    hi = __builtin_bit_cast(uint32_t, y);
  } else {
    const half2_t x = {(_Float16)v[0], (_Float16)v[1]}, y = {(_Float16)v[2], (_Float16)v[3]};
    lo = __builtin_bit_cast(uint32_t, x);
    hi = __builtin_bit_cast(uint32_t, y);
  }
  *reinterpret_cast<u32x2*>(a.out + elem) = u32x2{lo, hi};
}

// Two numbers to and from other workgroups: device-scope accesses, past the
// caches that are not coherent.
__device__ inline void put2(float* p, float x, float y) {
  const f32x2 v = {x, y};
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

__device__ inline f32x2 get2(const float* p) {
  return __builtin_bit_cast(f32x2, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT));
}

// A sequence of the call as the kernels see it.
struct Seq {
  int32_t c0, nq, len, first;   // first row of q, queries, tokens held, position of query 0
  Reach re;
  int32_t blocks;               // that any of its rows sees
};
// False (and nothing to do) for numbers that do not fit.
__device__ inline bool seq_from(const KvAttn& a, int c0, int c1, int len, Seq& s) {
  const int64_t nq = (int64_t)c1 - c0;
  s.blocks = 0;
  s.re = Reach{0, 0, 0};
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
  return true;
}

// Query of row r < 32 (up to 32 heads share a key/value head in the few-row kernel).
__device__ inline int query_of(const KvAttn& a, int r) { return (r * a.ratio_inv) >> 16; }

// Four channels of row r (sums v and of p, held times 2^base) and, once a row,
// the log of the sum of exponentials.
template <int D>
__device__ inline void answer4(const KvAttn& a, int c0, int head, int r, int c, const f32x4& v, float sum, float base) {
  const int qi = query_of(a, r), hh = r - qi * a.ratio;
  const int64_t o = (int64_t)(c0 + qi) * a.n_heads + head * a.ratio + hh;
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;   // 0: nothing seen; NaN stays
  store4(a, o * D + 4 * c, v * inv);
  if (a.lse && c == 0) a.lse[o] = (__builtin_amdgcn_logf(sum) - base) * kLn2;
}

// Work is a tile (sequence, head) or a part of one: tiles longer than `chunk`
// blocks are cut into equal parts, so that about kParts workgroups get work of
// like size whatever the lengths are. The parts of all tiles, sequence by
// sequence and head by head, are numbered by workgroup. A tile of n blocks is
// cut into sqrt(n) parts at most, since one workgroup joins them: the time of a
// part falls with their number and that of the join grows (131072 tokens of one
// head of 64 with 16 rows: 450 parts 72 us, 64 parts 30, 32 parts 38; 16384
// tokens of 8 heads of 128 with 4 rows: 64 parts 22.6, 23 parts 17.3).
struct Lanes {   // lane l: sequence base + l
  int32_t base, c0, nq, len, ns, w0, blocks;
};
__device__ inline void lanes_load(const KvAttn& a, uint32_t lane, int base, bool report, Lanes& l) {
  const int b = base + (int)lane;
  Seq s;
  s.c0 = s.nq = s.len = s.blocks = 0;
  s.re = Reach{0, 0, 0};
  if (b < a.batch && !seq_from(a, a.cu[b], a.cu[b + 1], a.lens[b], s)) {
    s.nq = 0;
    if (report) kv_flag(a.cache, VBQ_KV4_FLAG_LENGTH);
  }
  l.base = base;
  l.c0 = s.c0;
  l.nq = s.nq;
  l.len = s.len;
  l.ns = s.re.ns;
  l.w0 = s.re.w0;
  l.blocks = s.blocks;
}

// STAGES blocks a wavefront in LDS, STAGES - 1 of them on their way. Where
// registers allow four workgroups a CU (up to 8 rows, heads of up to 128), two
// stages: with heads of 128 the same bytes are on their way as with two
// workgroups of four stages, and the wavefronts hide each other's arithmetic
// (32 sequences of up to 8192 tokens, 4 rows a tile: 50 against 60 us). Eight
// wavefronts have two stages as well (8 x 4 queries of 4 heads a group, 20206
// tokens in all: 18.1 us, with four stages 19.5).
template <int G, int ROWS>
constexpr bool kRoomy = G <= 2 && ROWS <= 8;
typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));

template <int G, int ROWS, int STAGES>
__global__ __launch_bounds__((64 * kWaves<G, ROWS>), (kRoomy<G, ROWS>) ? 4 : G * ROWS > 64 ? 1 : 2) void k_kv4_attn(KvAttn a) {
  constexpr int WAVES = kWaves<G, ROWS>, D = 64 * G, PITCH = D + 4, BYTES = kKvGroupBytes * G;
  constexpr int NT = ROWS > 16 ? 2 : 1, COLS = ROWS > 16 ? 16 : ROWS;   // column tiles, and columns used of each
  constexpr int PARTS = 16 / COLS, PAIRS = 4 / PARTS;   // lanes that share a row's octet, token pairs of each
  constexpr int RING = WAVES * STAGES * BYTES, SUMS = WAVES * COLS * PITCH * 4;
  constexpr int JOIN = ROWS * kParts * 4 + 64 * WAVES * 16, AFTER = SUMS > JOIN ? SUMS : JOIN;
  // blocks; afterwards the wavefronts' sums, or the parts' factors and shares
  __shared__ __attribute__((aligned(16))) uint8_t ring[RING > AFTER ? RING : AFTER];
  __shared__ float wml[WAVES][ROWS][2];
  __shared__ uint32_t last;
  float* const buf = reinterpret_cast<float*>(ring);   // the wavefronts' sums, after a tile
  const uint32_t tid = threadIdx.x, lane = tid & 63u, col = lane & 15u, quarter = lane >> 4;
  const uint32_t qcol = col % COLS, part = col / COLS;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t* const own_ring = ring + wave * STAGES * BYTES;
  const uint32_t ring_lds = lds_addr(own_ring);

  // This workgroup's part: blocks i0 .. i1 - 1 of a tile.
  int b, head, i0 = 0, i1, blocks, c0, nq, len, part_no = 0, parts = 1;
  Reach re;
  if (a.parts) {
    Lanes ln;
    int total = 0;
    for (int base = 0; base < a.batch; base += 64) {
      lanes_load(a, lane, base, blockIdx.x == 0 && wave == 0, ln);
      total += __builtin_amdgcn_readlane(wave_scan(ln.blocks), 63);
      // sequences that see nothing have no parts: their rows are answered here
      for (uint64_t none = __ballot(ln.nq > 0 && ln.blocks == 0); none; none &= none - 1) {
        const int at = __builtin_ctzll(none);
        if ((uint32_t)(base + at) % gridDim.x != blockIdx.x) continue;
        const int n = __builtin_amdgcn_readlane(ln.nq, at) * a.n_heads;
        const int64_t from = (int64_t)__builtin_amdgcn_readlane(ln.c0, at) * a.n_heads;
        for (int e = (int)tid; e < n * (D / 4); e += 64 * WAVES) store4(a, from * D + 4 * e, f32x4{0.f, 0.f, 0.f, 0.f});
        if (a.lse)
          for (int e = (int)tid; e < n; e += 64 * WAVES) a.lse[from + e] = -__builtin_inff();
      }
    }
    const int chunk = max((int)(((uint32_t)total * (uint32_t)a.cache.heads + (uint32_t)a.parts - 1u) / (uint32_t)a.parts),
                          kLeastPart);
    int before = 0, incl, n, size;   // of each lane's sequence: parts up to its end, parts of a tile, blocks of a part
    uint64_t past;
    for (int base = 0;; base += 64) {
      if (a.batch > 64) lanes_load(a, lane, base, false, ln);
      const int most = max(chunk, (int)__builtin_amdgcn_sqrtf((float)ln.blocks));
      n = (int)((uint32_t)(ln.blocks + most - 1) / (uint32_t)most);
      size = n > 0 ? (int)((uint32_t)(ln.blocks + n - 1) / (uint32_t)n) : 1;   // nothing to see: no part
      n = (int)((uint32_t)(ln.blocks + size - 1) / (uint32_t)size);
      incl = before + wave_scan(n * a.cache.heads);
      past = __ballot(incl > (int)blockIdx.x);
      if (past) break;
      if (base + 64 >= a.batch) return;
      before = __builtin_amdgcn_readlane(incl, 63);
    }
    const int at = __builtin_ctzll(past);
    b = ln.base + at;
    blocks = __builtin_amdgcn_readlane(ln.blocks, at);
    c0 = __builtin_amdgcn_readlane(ln.c0, at);
    nq = __builtin_amdgcn_readlane(ln.nq, at);
    len = __builtin_amdgcn_readlane(ln.len, at);
    re.ns = __builtin_amdgcn_readlane(ln.ns, at);
    re.w0 = __builtin_amdgcn_readlane(ln.w0, at);
    parts = __builtin_amdgcn_readlane(n, at);
    const int rel = (int)blockIdx.x - (__builtin_amdgcn_readlane(incl, at) - parts * a.cache.heads);
    head = (int)((uint32_t)rel / (uint32_t)parts);
    part_no = rel - head * parts;
    i0 = part_no * __builtin_amdgcn_readlane(size, at);
    i1 = min(blocks, i0 + __builtin_amdgcn_readlane(size, at));
  } else {
    b = (int)(blockIdx.x / (uint32_t)a.cache.heads);
    head = (int)(blockIdx.x % (uint32_t)a.cache.heads);
    Seq sq;
    if (!seq_from(a, a.cu[b], a.cu[b + 1], a.lens[b], sq)) {
      if (tid == 0) kv_flag(a.cache, VBQ_KV4_FLAG_LENGTH);
      return;
    }
    c0 = sq.c0, nq = sq.nq, len = sq.len, re = sq.re, blocks = sq.blocks;
    if (nq == 0) return;
    i1 = blocks;
  }
  const int rows = nq * a.ratio, first = len - nq;
  const int p_min = a.causal ? first : len - 1, p_max = len - 1;   // positions of the rows

  // Queries, on their way while the first pages are looked up.
  u32x4 qraw[NT][G][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 16 * nt + (int)qcol;
    const int qi = query_of(a, r), hh = r - qi * a.ratio;
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
  uint64_t at = 0;   // lane i: where the wavefront's block i (of 64 at a time) lies
  uint64_t gone = 0, gone_before = 0;   // those that are not in the cache, and of the 64 before
  auto block_of = [&](int idx) { return idx < re.ns ? idx : idx - re.ns + re.w0; };
  auto start_copy = [&](int it) {
    if ((it & 63) == 0) {
      const int next = i0 + wave + WAVES * (it + (int)lane), blk = block_of(next);
      int page = 0;
      bool bad = false;
      if (next < i1) {
        page = a.table[(int64_t)b * a.width + (blk >> a.cache.block_shift)];
        bad = (uint32_t)page >= (uint32_t)a.cache.n_pages;
      }
      if (bad) {
        page = 0;   // copied, and left out of the sums
        kv_flag(a.cache, VBQ_KV4_FLAG_PAGE);
      }
      at = (uint64_t)kv_block(a.cache, G, (uint32_t)page, head, (uint32_t)blk & in_page);
      gone_before = gone;
      gone = __ballot(bad);
    }
    copy_block<G>(ring_lds + (uint32_t)(it % STAGES) * BYTES, lane_address(at, it & 63), lane);
  };
  const int count = i0 + wave < i1 ? (i1 - i0 - wave + WAVES - 1) / WAVES : 0;
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
    const int r = 16 * nt + (int)qcol;
    const bool in = r < rows;
    const int qi = query_of(a, r);
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
    to_log2[nt] = row_scale(a, ex - 13 + kCodeExp);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const _Float16 v0 = (_Float16)(x[g][st][i] * up), v1 = (_Float16)(x[g][st][i + 4] * up);
          sum += (float)v0 + (float)v1;
          qf[nt][g][st][2 * i] = v0;
          qf[nt][g][st][2 * i + 1] = v1;
        }
      qsum[nt][g] = ldexpf(rows_sum(sum), -kCodeExp);
    }
    const int p = a.causal ? first + qi : len - 1;
    hi[nt] = in ? min(p, len - 1) : -1;
    lo[nt] = a.window ? max(p, 0) - a.window + 1 : INT32_MIN;   // (rows before position 0 see nothing)
  }

  // Running maximum m, and sums held times 2^base, base = S - m: of p, of p o,
  // and (times 2^-kCodeExp) of p s code.
  float m[NT], base[NT], l[NT], po[NT][G];
  f32x4 acc[NT][G][4];
  float mul[NT], add[NT];   // of a score on its way to exp2
  bool far = false;         // a row of the wavefront has its maximum far out
  float shift[NT];   // S of the lane's row
  int limit[NT];     // largest scale that S is fit for (bits of an fp16)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    shift[nt] = 0.f;
    limit[nt] = -1;
    m[nt] = kNoMax;
    base[nt] = -kNoMax;
    mul[nt] = to_log2[nt];
    add[nt] = base[nt];
    l[nt] = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      po[nt][g] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) acc[nt][g][w] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
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
    if ((gone | gone_before) && ((((it ^ min(ahead, count - 1)) >> 6 ? gone_before : gone) >> (it & 63)) & 1u)) continue;
    const int blk = block_of(i0 + wave + WAVES * it);
    const uint8_t* const k = own_ring + (it % STAGES) * BYTES;

    // Scores of the lane's tokens 8 quarter + PAIRS part + j (+ 4).
    const int t0 = blk * kKvBlock, mine = t0 + 8 * (int)quarter + PAIRS * (int)part;
    float sc[NT][PAIRS][2];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const u32x4 kc = lds16(k + 1024 * g + 16 * lane);
      const uint8_t* const so = k + kv_key_so(G) + 128 * g + 16 * quarter + 2 * PAIRS * part;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const half8_t a0 = codes_of(kc[2 * h]), a1 = codes_of(kc[2 * h + 1]);
        const Halves<PAIRS> s(so + 8 * h), o(so + 64 + 8 * h);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f32x4 d = f32x4{0.f, 0.f, 0.f, 0.f};
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, qf[nt][g][0], d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, qf[nt][g][1], d, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < PAIRS; ++j) {
            float x = d[j];
            if constexpr (PARTS == 2) x = part ? d[2 + j] : d[j];
            if constexpr (PARTS == 4) {
              const float x0 = part & 1u ? d[1] : d[0], x1 = part & 1u ? d[3] : d[2];
              x = part & 2u ? x1 : x0;
            }
            x = __builtin_fmaf(s[j], x, o[j] * qsum[nt][g]);
            sc[nt][j][h] = g ? sc[nt][j][h] + x : x;
          }
        }
      }
    }
    // Values' scales and offsets, pairs (j, j + 4).
    uint32_t vs[G][PAIRS], vo[G][PAIRS];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint8_t* const so = k + kv_value_so(G) + 128 * g + 16 * quarter + 4 * PAIRS * part;
      const Halves<2 * PAIRS> s(so), o(so + 64);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        vs[g][j] = s.w[j];
        vo[g][j] = o.w[j];
      }
    }
    if (t0 + kKvBlock > len) {   // places past the sequence's end may hold anything
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        const uint32_t keep = mine + j + 4 < len ? 0xFFFFFFFFu : mine + j < len ? 0x0000FFFFu : 0u;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          vs[g][j] &= keep;
          vo[g][j] &= keep;
        }
      }
    }
    // The largest scale among the tokens that the lane's row sees.
    int s_max[NT];
    const bool edge = t0 + kKvBlock - 1 > min(p_min, len - 1) ||
                      (a.window && t0 <= p_max - a.window && t0 + kKvBlock > a.sinks);
    if (edge) {   // not every row sees all of the block
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        ushort2_t top = {0, 0};
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
          uint32_t keep = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int t = mine + j + 4 * h;
            const bool see = t <= hi[nt] && (t >= lo[nt] || t < a.sinks);
            sc[nt][j][h] = see ? sc[nt][j][h] : -__builtin_inff();
            keep |= see ? 0xFFFFu << (16 * h) : 0u;
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t u = vs[g][j] & keep;
            top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2_t, u));
          }
        }
        s_max[nt] = max((int)top.x, (int)top.y);
      }
    } else {
      ushort2_t top = {0, 0};
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
          const uint32_t u = vs[g][j];
          top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2_t, u));
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s_max[nt] = max((int)top.x, (int)top.y);
    }

    // Running maximum; sums follow it and S.
    bool grow = false;
    float mt[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float t = sc[nt][0][0];
#pragma unroll
      for (int j = 0; j < PAIRS; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) t = fmaxf(t, sc[nt][j][h]);
      mt[nt] = fmaxf(m[nt], lanes_max<PARTS>(t) * to_log2[nt]);
      grow |= mt[nt] > m[nt] || s_max[nt] > limit[nt];
    }
    if (__any(grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // S brings the row's largest scale s below 2^12, and stays fit up to 8 s.
        const float top = lanes_max<PARTS>((float)__builtin_bit_cast(_Float16, (uint16_t)s_max[nt]));
        if ((int)__builtin_bit_cast(uint16_t, (_Float16)top) > limit[nt]) {
          const int ex = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 126;   // top < 2^ex
          shift[nt] = top > 0.f ? (float)(12 - ex) : 0.f;
          const _Float16 most = (_Float16)fminf(ldexpf(1.f, ex + 3), 65504.f);
          limit[nt] = top > 0.f ? (int)__builtin_bit_cast(uint16_t, most) : 0;
        }
        m[nt] = mt[nt];
        const float now = shift[nt] - mt[nt], f = __builtin_amdgcn_exp2f(now - base[nt]);
        base[nt] = now;
        l[nt] *= f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          po[nt][g] *= f;
#pragma unroll
          for (int w = 0; w < 4; ++w) acc[nt][g][w] *= f;
        }
      }
      bool out = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) out |= is_far(m[nt]);
      far = __any(out);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mul[nt] = far ? 1.f : to_log2[nt];
        add[nt] = far ? shift[nt] : base[nt];
      }
    }
    if (far) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) sc[nt][j][h] = below(sc[nt][j][h], to_log2[nt], m[nt]);
    }
    // Probabilities times 2^S.
    float p[NT][PAIRS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) p[nt][j][h] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[nt][j][h], mul[nt], add[nt]));
        l[nt] += p[nt][j][0] + p[nt][j][1];
      }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      half8_t big[NT], small[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t x[PAIRS], y[PAIRS];
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
          const half2_t s = pair_of(vs[g][j]), o = pair_of(vo[g][j]);
          const float u0 = p[nt][j][0] * (float)s.x, u1 = p[nt][j][1] * (float)s.y;
          const half2_t b = {(_Float16)u0, (_Float16)u1};
          const half2_t r = {(_Float16)(u0 - (float)b.x), (_Float16)(u1 - (float)b.y)};
          x[j] = __builtin_bit_cast(uint32_t, b);
          y[j] = __builtin_bit_cast(uint32_t, r);
          po[nt][g] = __builtin_fmaf(p[nt][j][0], (float)o.x, __builtin_fmaf(p[nt][j][1], (float)o.y, po[nt][g]));
        }
        // The octet's four pairs, from the lanes that hold them, in column `qcol`.
        u32x4 bx, by;
        if constexpr (PARTS == 1) {
          bx = u32x4{x[0], x[1], x[2], x[3]};
          by = u32x4{y[0], y[1], y[2], y[3]};
        } else if constexpr (PARTS == 2) {
          bx = u32x4{x[0], x[1], row_down<8>(x[0]), row_down<8>(x[1])};
          by = u32x4{y[0], y[1], row_down<8>(y[0]), row_down<8>(y[1])};
        } else {
          bx = u32x4{x[0], row_down<4>(x[0]), row_down<8>(x[0]), row_down<12>(x[0])};
          by = u32x4{y[0], row_down<4>(y[0]), row_down<8>(y[0]), row_down<12>(y[0])};
        }
        big[nt] = __builtin_bit_cast(half8_t, bx);
        small[nt] = __builtin_bit_cast(half8_t, by);
      }
      const u32x4 vc = lds16(k + kv_value_codes(G) + 1024 * g + 16 * lane);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const half8_t v = codes_of(vc[w]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][g][w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, big[nt], acc[nt][g][w], 0, 0, 0);
          acc[nt][g][w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, small[nt], acc[nt][g][w], 0, 0, 0);
        }
      }
    }
  }

  // Join the wavefronts: every one scales its sums to the smallest base.
  float sum_l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    sum_l[nt] = lanes_sum<PARTS>(l[nt]);
#pragma unroll
    for (int g = 0; g < G; ++g) po[nt][g] = lanes_sum<PARTS>(po[nt][g]);
    if (quarter == 0 && part == 0) {
      wml[wave][16 * nt + qcol][0] = base[nt];
      wml[wave][16 * nt + qcol][1] = sum_l[nt];
    }
  }
  __syncthreads();
  float* const slot = a.acc + (int64_t)blockIdx.x * ROWS * D;   // a part's sums, and their bases and sums of p
  float* const slot_ml = a.ml + (int64_t)blockIdx.x * ROWS * 2;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (16 * nt >= rows) break;
    if (nt) __syncthreads();   // the buffer is taken again
    if (part == 0) {
      const int rr = 16 * nt + (int)qcol;
      float low = wml[0][rr][0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) low = fminf(low, wml[w][rr][0]);
      const float f = __builtin_amdgcn_exp2f(low - base[nt]), f_code = ldexpf(f, kCodeExp);
      float* const to = buf + (wave * COLS + qcol) * PITCH + 16 * quarter;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float z = po[nt][g] * f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 v = {__builtin_fmaf(acc[nt][g][0][i], f_code, z), __builtin_fmaf(acc[nt][g][1][i], f_code, z),
                           __builtin_fmaf(acc[nt][g][2][i], f_code, z), __builtin_fmaf(acc[nt][g][3][i], f_code, z)};
          *reinterpret_cast<f32x4*>(to + 64 * g + 4 * i) = v;
        }
      }
    }
    __syncthreads();
    for (int e = (int)tid; e < COLS * (D / 4); e += 64 * WAVES) {
      const int row = e / (D / 4), c = e % (D / 4), rr = 16 * nt + row;
      if (rr >= rows) break;
      float low = wml[0][rr][0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) low = fminf(low, wml[w][rr][0]);
      float sum = 0.f;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        sum += wml[w][rr][1] * __builtin_amdgcn_exp2f(low - wml[w][rr][0]);
        v += *reinterpret_cast<const f32x4*>(buf + (w * COLS + row) * PITCH + 4 * c);
      }
      if (parts == 1) {
        answer4<D>(a, c0, head, rr, c, v, sum, low);
      } else {
        put2(slot + rr * D + 4 * c, v[0], v[1]);
        put2(slot + rr * D + 4 * c + 2, v[2], v[3]);
        if (c == 0) put2(slot_ml + 2 * rr, low, sum);
      }
    }
  }
  if (parts == 1) return;

  // Join the tile's parts. The sums above are device-scope stores, which write
  // through the caches; each wavefront waits for its own before the barrier, so
  // once the tile's counter counts this part every workgroup's device-scope
  // loads see them. The part that is counted last joins all of them, in order,
  // and sets the counter back. (An acquire fence and ordinary loads instead: 33
  // against 22 us for 256 tiles of 34 blocks, since every fence empties an L2.)
  uint32_t* const counter = a.counters + (b * a.cache.heads + head);
  __builtin_amdgcn_s_waitcnt(VBQ_VMCNT_IMM(0));
  __syncthreads();
  if (tid == 0) {
    last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(parts - 1);
    if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  const float* const acc0 = slot - (int64_t)part_no * ROWS * D;
  const float* const ml0 = slot_ml - (int64_t)part_no * ROWS * 2;
  float* const factor = buf;                                                 // [rows][kParts]
  f32x4* const share = reinterpret_cast<f32x4*>(ring + ROWS * kParts * 4);   // [threads]
  constexpr int THREADS = 64 * WAVES, ROW_LANES = ROWS < 16 ? 16 : THREADS / ROWS;
  {   // some lanes a row: the smallest base, each part's factor, the sum
    const int row = (int)tid / ROW_LANES, j = (int)tid % ROW_LANES;
    float low = -kNoMax, sum = 0.f;   // sum is held times 2^low
    if (row < rows) {
      for (int p0 = j; p0 < parts; p0 += 8 * ROW_LANES) {
        f32x2 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i == 0 || p0 - j + i * ROW_LANES < parts)
            v[i] = get2(ml0 + (min(p0 + i * ROW_LANES, parts - 1) * ROWS + row) * 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int p = p0 + i * ROW_LANES;
          if (p >= parts) break;
          factor[row * kParts + p] = v[i].x;
          const float to = fminf(low, v[i].x);
          sum = __builtin_fmaf(sum, __builtin_amdgcn_exp2f(to - low), v[i].y * __builtin_amdgcn_exp2f(to - v[i].x));
          low = to;
        }
      }
    }
    const float own = low;
#pragma unroll
    for (int d = 1; d < ROW_LANES; d <<= 1) low = fminf(low, __shfl_xor(low, d, 64));
    sum *= __builtin_amdgcn_exp2f(low - own);
    if (row < rows)
      for (int p = j; p < parts; p += ROW_LANES)
        factor[row * kParts + p] = __builtin_amdgcn_exp2f(low - factor[row * kParts + p]);
#pragma unroll
    for (int d = 1; d < ROW_LANES; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if (j == 0 && row < rows) {
      wml[0][row][0] = low;
      wml[0][row][1] = sum;
    }
  }
  __syncthreads();
  // Threads beyond the rows' outputs share the parts. A thread's loads go out
  // together, 16 at a time (where a thread's part is past the last, the last is
  // read and left out): one by one they took 6 of 28 us for 64 tiles of 20 rows
  // in 4 parts.
  constexpr int ROUNDS = (ROWS * D / 4 + THREADS - 1) / THREADS, BATCH = 16 / ROUNDS;   // (the last one may be ragged)
  static_assert(ROUNDS * THREADS >= ROWS * D / 4 && BATCH >= 1, "every output of a tile has a thread and a round");
  const int ne = rows * (D / 4), shares = ne <= THREADS / 2 ? THREADS / ne : 1;
  const int e0 = shares > 1 ? (int)tid % ne : (int)tid, share_no = shares > 1 ? (int)tid / ne : 0;
  f32x4 v[ROUNDS];
  const float* from[ROUNDS];
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    v[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int e = min(e0 + k * THREADS, ne - 1);
    from[k] = acc0 + e / (D / 4) * D + 4 * (e % (D / 4));
  }
  if (share_no < shares)
    for (int p0 = share_no; p0 < parts; p0 += BATCH * shares) {
      f32x2 x[BATCH][ROUNDS], y[BATCH][ROUNDS];
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
          if (i && p0 - share_no + i * shares >= parts) continue;
          const float* const q = from[k] + min(p0 + i * shares, parts - 1) * (ROWS * D);
          x[i][k] = get2(q);
          y[i][k] = get2(q + 2);
        }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int p = p0 + i * shares;
        if (p >= parts) break;
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k)
          v[k] += f32x4{x[i][k].x, x[i][k].y, y[i][k].x, y[i][k].y} *
                  factor[min(e0 + k * THREADS, ne - 1) / (D / 4) * kParts + p];
      }
    }
  if (shares > 1) {   // (then a thread has one output at most: ne <= THREADS / 2)
    share[tid] = v[0];
    __syncthreads();
    if (share_no == 0)
      for (int i = 1; i < shares; ++i) v[0] += share[e0 + i * ne];
  }
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const int e = e0 + k * THREADS, row = e / (D / 4);
    if (e < ne && share_no == 0) answer4<D>(a, c0, head, row, e % (D / 4), v[k], wml[0][row][1], wml[0][row][0]);
  }
}

// ---- many rows ---------------------------------------------------------------------
// Four wavefronts take 32 rows each of one head and walk the blocks together. A
// block is copied raw to LDS, spread there into operands (a quarter by each
// wavefront), and multiplied by every wavefront with 32x32x16 MFMAs: S^T = K
// Q^T, O^T = V^T P^T. One turn of the loop spreads the keys of block i + 2 and
// the values of block i + 1, forms the scores of block i + 1 and the
// probabilities and output of block i, in one straight piece of code, so that
// matrix and vector instructions overlap. Key operands are the exact codes as
// normal fp16 numbers, of whose products the matrix unit loses nothing that fp32
// holds (see above): a word is spread once for 128 rows, and 2048 queries over
// 10240 tokens take 1% longer so than with c 2^-20. Scores take scale in fp32 as
// above and offsets by one more MFMA: A holds a token's offsets o_g, B the rows'
// sums of q over group g. Rounding keys to fp16 instead would save the scaling,
// but a score's error is multiplied into its probability: it doubled the
// output's error in fp16. Values are s c + o rounded once to fp16 (as codes they
// would need p s of every group and what its rounding leaves, 2 G conversions a
// probability instead of one, where vector instructions bound the kernel), as are
// probabilities; for fp16 outputs (FINE) what is left of a probability is
// multiplied too: without it the outputs of 2500 rows under a window of 500
// were off by 3.2e-4 (relative, whole tensor), with it by 2.8e-4, of which
// 2.1e-4 are the rounding of the output itself; bf16 outputs are off by 1.7e-3
// either way.
//   Bounds. 2048 bf16 queries of 32 heads of 128 over 10240 tokens: 309 GFLOP in
// 426 us, 0.73 PFLOP/s (a library product of 8192^3 reaches 1.24 to 1.37; some
// cards run the same code in 480 us). A turn of one wavefront is 17 MFMAs (544
// cycles), about 150 vector instructions (850 cycles) and 28 KB of LDS reads (220
// cycles of the CU, times 8 wavefronts), and two wavefronts a SIMD overlap them
// in part. With values spread a block
// later than keys two buffers do for both, and heads of 192 fit twice on a CU (17 x
// 1193 queries, 16 heads: 462 -> 317 us). Heads of 256 have registers for one
// wavefront a SIMD: 3 sequences under a window of 500, 36 GFLOP in 150 us;
// 2.2 us a block, 7 us before the first and 2 us after the last, and 630
// workgroups on 256 CUs end in a third round. (64 rows a wavefront: 536 against
// 447 us. Reads of a group ahead of its products, held there by scheduling
// barriers: no change.)
// In LDS keys and values lie as the operands are read, 16 bytes a lane:
//   keys:   chunk (channel / 8, row R), the 8 channels as pairs (n, n + 4);
//           token 8 (2 A + h) + 4 u + b is row 8 (2 A + u) + 4 h + b, so the
//           score MFMA leaves octet 2 A + h whole in lane half h;
//   values: chunk (octet / 2, channel tile T, octet % 2, row), the octet's
//           tokens as pairs; channel 64 g + 4 m + w is row 16 (w % 2) + m of
//           tile 2 g + w / 2, so a result holds 16 neighbouring channels a lane.
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kTileShift = 7.f;   // probabilities are held times 2^7 ...
constexpr float kTileSlack = 8.f;   // ... and the maximum may be passed by 2^8 before sums are scaled

// Eight codes of a word as normal fp16 numbers c 2^-kTileCodeExp, pairs (n, n + 4).
constexpr int kTileCodeExp = 10;
__device__ inline half8_t normal_codes_of(uint32_t w) {
  const half2_t up = {(_Float16)0x1p14f, (_Float16)0x1p14f}, up4 = {(_Float16)0x1p10f, (_Float16)0x1p10f};
  const uint32_t h = w >> 8;
  u32x4 r;
  r.x = __builtin_bit_cast(uint32_t, pair_of(w & 0x000F000Fu) * up);
  r.y = __builtin_bit_cast(uint32_t, pair_of(w & 0x00F000F0u) * up4);
  r.z = __builtin_bit_cast(uint32_t, pair_of(h & 0x000F000Fu) * up);
  r.w = __builtin_bit_cast(uint32_t, pair_of(h & 0x00F000F0u) * up4);
  return __builtin_bit_cast(half8_t, r);
}

// Constants of the decode, opaque to the compiler: with the masks in scalar and
// the exponent in a vector register (w & mask) | exponent is one instruction;
// known constants become two with a literal each.
struct Decode {
  uint32_t m0, m4, ex;
  __device__ Decode() : m0(0x000F000Fu), m4(0x00F000F0u), ex(0x64006400u) {
    asm("" : "+s"(m0));
    asm("" : "+s"(m4));
    asm("" : "+v"(ex));
  }
};
// Eight values s c + o of a word as pairs (n, n + 4), one rounding each: the
// codes are made exact by an exponent that is subtracted again.
__device__ inline u32x4 values_of(const Decode& dc, uint32_t w, const half2_t (&s)[4], const half2_t (&o)[4]) {
  const half2_t one = {(_Float16)1024.f, (_Float16)1024.f}, sx = {(_Float16)0.0625f, (_Float16)0.0625f},
                sb = {(_Float16)-64.f, (_Float16)-64.f};
  const uint32_t h = w >> 8;
  const half2_t c[4] = {pair_of((w & dc.m0) | dc.ex) - one,
                        __builtin_elementwise_fma(pair_of((w & dc.m4) | dc.ex), sx, sb),
                        pair_of((h & dc.m0) | dc.ex) - one,
                        __builtin_elementwise_fma(pair_of((h & dc.m4) | dc.ex), sx, sb)};
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c[i], s[i], o[i]));
  return r;
}

__device__ inline float half_max(float v) {   // with the lane 32 apart
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const pair_t p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t x = p.x, y = p.y;
  return fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
__device__ inline float half_sum(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const pair_t p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t x = p.x, y = p.y;
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Blocks that a tile's rows r0 .. look at, and how many of them a part takes.
constexpr int kRowTile = 128;
__device__ inline Reach tile_reach(const KvAttn& a, const Seq& sq, int rows, int r0) {
  const int r1 = min(rows, r0 + kRowTile);
  return reach(sq.len, a.causal ? sq.first + r0 / a.ratio : sq.len - 1,
               a.causal ? sq.first + (r1 - 1) / a.ratio : sq.len - 1, a.window, a.sinks);
}
constexpr int kLeastTilePart = 8, kTileParts = 64;
__device__ inline int part_blocks(const KvAttn& a, const Reach& re) {
  return max((int)((uint32_t)(re.ns + re.nw + a.parts - 1) / (uint32_t)a.parts), kLeastTilePart);
}

template <int G, bool FINE>
__global__ __launch_bounds__(256, G >= 4 ? 1 : 2) void k_kv4_attn_tile(KvAttn a) {
  constexpr int WAVES = 4, ROWS = kRowTile, D = 64 * G, BYTES = kKvGroupBytes * G, RAW = 4, TILES = D / 32;
  constexpr int SHARE = BYTES / WAVES;   // a wavefront's part of a block's copy
  constexpr int COPIES = (SHARE + 1023) / 1024;
  constexpr int HELD = 32 * D * 2;   // a block's keys, or values
  static_assert(SHARE % 16 == 0, "copies are 16 bytes a lane");
  __shared__ __attribute__((aligned(16))) uint8_t raw[RAW * BYTES];
  __shared__ __attribute__((aligned(16))) uint8_t keys[2 * HELD], vals[2 * HELD];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, col = lane & 31u, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t raw_lds = lds_addr(raw);
  const Decode dc;

  // The tiles of a (sequence, head) lie a multiple of the heads apart (one L2
  // where that is a multiple of 8); the last rows, which see most, go first.
  const uint32_t bh_n = (uint32_t)(a.batch * a.cache.heads);
  const uint32_t bh = blockIdx.x % bh_n;
  const int b = (int)(bh / (uint32_t)a.cache.heads), head = (int)(bh % (uint32_t)a.cache.heads);
  Seq sq;
  if (!seq_from(a, a.cu[b], a.cu[b + 1], a.lens[b], sq)) {
    if (tid == 0) kv_flag(a.cache, VBQ_KV4_FLAG_LENGTH);
    return;
  }
  const int rows = sq.nq * a.ratio, rts = (rows + ROWS - 1) / ROWS;
  const int rt = rts - 1 - (int)(blockIdx.x / bh_n);
  if (rt < 0) return;
  const int len = sq.len, first = sq.first;
  const int r0 = rt * ROWS;
  const Reach re = tile_reach(a, sq, rows, r0);
  // this workgroup's part: blocks i0 .. i0 + blocks - 1 of the tile
  const int per = part_blocks(a, re), i0 = (int)blockIdx.y * per;
  const int blocks = min(re.ns + re.nw - i0, per);
  const bool whole = re.ns + re.nw <= per;
  if (i0 && blocks <= 0) return;
  auto block_of = [&](int i) { return i0 + i < re.ns ? i0 + i : i0 + i - re.ns + re.w0; };

  // Copies: lane i keeps the page of block i of 64.
  const uint32_t in_page = (1u << a.cache.block_shift) - 1u;
  uint64_t where = 0;   // lane i: where block i of 64 lies
  uint64_t gone = 0, gone_before = 0;   // blocks of the 64 (and of those before) whose page is not in the cache
  auto start_copy = [&](int i) {
    if ((i & 63) == 0) {
      const int next = i + (int)lane, blk = block_of(next);
      int page = 0;
      bool bad = false;
      if (next < blocks) {
        page = a.table[(int64_t)b * a.width + (blk >> a.cache.block_shift)];
        bad = (uint32_t)page >= (uint32_t)a.cache.n_pages;
      }
      if (bad) {
        page = 0;   // copied, and hidden
        if (wave == 0) kv_flag(a.cache, VBQ_KV4_FLAG_PAGE);
      }
      where = (uint64_t)kv_block(a.cache, G, (uint32_t)page, head, (uint32_t)blk & in_page) + wave * SHARE;
      gone_before = gone;
      gone = __ballot(bad);
    }
    const u32x4 rsrc = make_rsrc(lane_address(where, i & 63), SHARE);
    const uint32_t to = raw_lds + (uint32_t)(i % RAW) * BYTES + (uint32_t)wave * SHARE;
#pragma unroll
    for (int c = 0; c < SHARE / 1024; ++c) dma16(rsrc, to + 1024 * c, 1024 * c + 16 * lane);
    if (lane < (SHARE % 1024) / 16) dma16(rsrc, to + SHARE / 1024 * 1024, SHARE / 1024 * 1024 + 16 * lane);
  };
  auto is_gone = [&](int i, int newest) {   // newest: the last block whose copy was started
    if (!(gone | gone_before)) return false;
    return (bool)((((i ^ newest) >> 6 ? gone_before : gone) >> (i & 63)) & 1u);
  };

  // Queries: B operands, channels of a chunk as pairs; what the lane's row sees.
  for (int i = 0; i < 2; ++i)
    if (i < blocks) start_copy(i);
  half8_t qf[D / 16], qsum;
  float to_log2;
  int hi, lo;
  const int w_r0 = r0 + 32 * wave;   // the wavefront's first row
  {
    const int r = w_r0 + (int)col, qi = r / a.ratio, hh = r - qi * a.ratio;
    u32x4 x[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      x[c] = u32x4{0, 0, 0, 0};
      if (r < rows)
        x[c] = *reinterpret_cast<const u32x4*>(a.q + (int64_t)(sq.c0 + qi) * a.q_ts +
                                               (int64_t)(head * a.ratio + hh) * a.q_hs + 16 * c + 8 * half);
    }
    // (one branch on the type, not one a number)
    float y[D / 16][8];
    if (a.bf16) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[c][2 * i] = __builtin_bit_cast(float, x[c][i] << 16);
          y[c][2 * i + 1] = __builtin_bit_cast(float, x[c][i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = x[c][i];
          y[c][2 * i] = (float)pair_of(u).x;
          y[c][2 * i + 1] = (float)pair_of(u).y;
        }
    }
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[c][i]));
    top = half_max(top);
    int ex = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
    ex = top > 0.f ? max(ex, -100) : 13;
    const float up = ldexpf(1.f, 13 - ex);
    to_log2 = row_scale(a, ex - 13 + kTileCodeExp);
#pragma unroll
    for (int j = 0; j < 8; ++j) qsum[j] = (_Float16)0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int c = 4 * g; c < 4 * g + 4; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const _Float16 v0 = (_Float16)(y[c][i] * up), v1 = (_Float16)(y[c][i + 4] * up);
          sum += (float)v0 + (float)v1;
          qf[c][2 * i] = v0;
          qf[c][2 * i + 1] = v1;
        }
      // the sum as two fp16 numbers, which leave 2^-25 at most of it (the row's largest |q| is 2^3 or more here)
      sum = ldexpf(half_sum(sum), -kTileCodeExp);
      const _Float16 big = (_Float16)sum;
      qsum[2 * g] = big;
      qsum[2 * g + 1] = (_Float16)(sum - (float)big);
    }
    const int p = a.causal ? first + qi : len - 1;
    hi = r < rows ? min(p, len - 1) : -1;
    lo = a.window ? max(p, 0) - a.window + 1 : INT32_MIN;
  }
  // this wavefront's first and last positions
  const int w_r1 = min(rows, w_r0 + 32);
  const int w_min = min(a.causal ? first + w_r0 / a.ratio : len - 1, len - 1);
  const int w_max = w_r0 >= rows ? -1 : a.causal ? max(first + (w_r1 - 1) / a.ratio, -1) : len - 1;

  // Operands of block i: a wavefront takes word `wave` of every lane's four.
  const uint32_t m16 = lane & 15u, kq = lane >> 4;
  auto spread_keys = [&](int i) {
    const uint8_t* const from = raw + (i % RAW) * BYTES + 16 * lane + 4 * wave;
    uint8_t* const to = keys + (i & 1) * HELD + ((4 * (wave & 1) + kq) * 32 + 16 * (m16 >> 3) + 8 * (wave >> 1) +
                                                 (m16 & 7u)) * 16;
#pragma unroll
    for (int g = 0; g < G; ++g)
      *reinterpret_cast<half8_t*>(to + 8 * 32 * 16 * g) =
          normal_codes_of(*reinterpret_cast<const uint32_t*>(from + 1024 * g));
  };
  auto spread_values = [&](int i) {
    const uint8_t* const from = raw + (i % RAW) * BYTES;
    uint8_t* const to =
        vals + (i & 1) * HELD + (((kq >> 1) * TILES + (wave >> 1)) * 64 + 32 * (kq & 1u) + 16 * (wave & 1) + m16) * 16;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(from + kv_value_codes(G) + 1024 * g + 16 * lane + 4 * wave);
      const Halves<8> s(from + kv_value_so(G) + 128 * g + 16 * kq), o(from + kv_value_so(G) + 128 * g + 64 + 16 * kq);
      const half2_t s2[4] = {pair_of(s.w[0]), pair_of(s.w[1]), pair_of(s.w[2]), pair_of(s.w[3])};
      const half2_t o2[4] = {pair_of(o.w[0]), pair_of(o.w[1]), pair_of(o.w[2]), pair_of(o.w[3])};
      *reinterpret_cast<u32x4*>(to + 2 * 64 * 16 * g) = values_of(dc, w, s2, o2);
    }
  };
  // Places of block i past the sequence's end (all of them if its page is not
  // in the cache) may hold anything: their values' scales and offsets become 0.
  auto blank = [&](int i, int end) {
    if (tid < 32 * G) {
      const int t = (int)(tid & 31u);
      const uint32_t place = 8 * ((uint32_t)t >> 3) + 2 * (t & 3) + ((t & 7) >> 2);
      _Float16* const so = reinterpret_cast<_Float16*>(raw + (i % RAW) * BYTES + kv_value_so(G) + 128 * (tid >> 5));
      if (t >= end) so[place] = so[32 + place] = (_Float16)0.f;
    }
  };
  // Scores of block i, unscaled by to_log2 and unmasked: register 8 A + 4 u + b
  // is token 8 (2 A + half) + 4 u + b.
  const uint32_t tok = 16 * (col >> 4) + 8 * ((col >> 2) & 1u) + 4 * ((col >> 3) & 1u) + (col & 3u);   // of row `col`
  f32x16 none;
#pragma unroll
  for (int j = 0; j < 16; ++j) none[j] = 0.f;
  auto scores = [&](int i, f32x16& x) {
    const uint8_t* const k = keys + (i & 1) * HELD;
    const uint8_t* const so = raw + (i % RAW) * BYTES + kv_key_so(G);
    half8_t off;
#pragma unroll
    for (int j = 0; j < 8; ++j) off[j] = (_Float16)0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const _Float16 o = *reinterpret_cast<const _Float16*>(so + 128 * g + 64 + 2 * tok);
      off[2 * g] = off[2 * g + 1] = half ? (_Float16)0.f : o;
    }
    x = __builtin_amdgcn_mfma_f32_32x32x16_f16(off, qsum, none, 0, 0, 0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      f32x16 d;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const half8_t kc = __builtin_bit_cast(half8_t, lds16(k + 1024 * (4 * g + c) + 16 * lane));
        d = __builtin_amdgcn_mfma_f32_32x32x16_f16(kc, qf[4 * g + c], c ? d : none, 0, 0, 0);
      }
#pragma unroll
      for (int A = 0; A < 2; ++A) {
        const Halves<8> s(so + 128 * g + 16 * (2 * A + half));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[8 * A + j] = __builtin_fmaf(s[j], d[8 * A + j], x[8 * A + j]);
      }
    }
  };

  // Running maximum, sum of p times 2^(kTileShift - m), sums of p v; mx: a block's maximum.
  float m = kNoMax, l = 0.f, mx;
  bool far = false;   // a row of the wavefront has its maximum far out
  f32x16 acc[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) acc[t] = none;
  // Masks scores of block i; their rows' maxima, and whether one passes its
  // running maximum by more than the slack.
  auto settle = [&](int i, bool hidden, f32x16& sc) {
    const int t0 = block_of(i) * kKvBlock;
    if (hidden || t0 + kKvBlock - 1 > w_min || (a.window && t0 <= w_max - a.window && t0 + kKvBlock > a.sinks)) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int t = t0 + 8 * (2 * (j >> 3) + (int)half) + (j & 7);
        const bool see = !hidden && t <= hi && (t >= lo || t < a.sinks);
        sc[j] = see ? sc[j] : -__builtin_inff();
      }
    }
    float top = sc[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) top = fmaxf(top, sc[j]);
    mx = half_max(top) * to_log2;
    return (bool)__any(mx > m + kTileSlack);
  };
  // Waits for the copy of block i (of which at most block i + 1's follow), for
  // every wavefront, and starts block i + 2's.
  auto arrive = [&](int i) {
    if (i + 1 < blocks)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(COPIES) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    if (i < blocks) {
      const int end = is_gone(i, min(i + 1, blocks - 1)) ? 0 : len - block_of(i) * kKvBlock;
      if (end < kKvBlock) {
        blank(i, end);
        __syncthreads();
      }
      if (i + 2 < blocks) start_copy(i + 2);
    }
  };

  if (blocks > 0) {
    arrive(0);
    spread_keys(0);
    spread_values(0);
    arrive(1);
    bool hide = is_gone(0, min(2, blocks - 1));
    if (blocks > 1) spread_keys(1);
    f32x16 sc;
    scores(0, sc);
    settle(0, hide, sc);
    // The inner loop runs while no row's scores pass its running maximum by
    // more than the slack: it has no vector arithmetic on the sums, so they
    // stay in accumulation registers.
    auto settle_far = [&]() {
#pragma unroll
      for (int j = 0; j < 16; ++j) sc[j] = below(sc[j], to_log2, m);
    };
    for (int i = 0; i < blocks;) {
      const float mt = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - mt);
      m = mt;
      far = __any(is_far(m));
      if (far) settle_far();
      const float mul = far ? 1.f : to_log2, base = far ? kTileShift : kTileShift - m;
      l *= f;
#pragma unroll
      for (int t = 0; t < TILES; ++t) acc[t] *= f;
      bool pass = false;
      do {
        arrive(i + 2);
        hide = i + 1 < blocks && is_gone(i + 1, min(i + 4, blocks - 1));
        // (the last turns spread and score what an older block left: unused)
        f32x16 next;
        scores(i + 1, next);
        half8_t pf[2], pl[2];   // probabilities, and what their rounding leaves
        const half2_t ones = {(_Float16)1.f, (_Float16)1.f};
#pragma unroll
        for (int A = 0; A < 2; ++A)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[8 * A + j], mul, base));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[8 * A + 4 + j], mul, base));
            const half2_t pr = {(_Float16)p0, (_Float16)p1};
            pf[A][2 * j] = pr.x;
            pf[A][2 * j + 1] = pr.y;
            if constexpr (FINE) {
              l += p0 + p1;
              pl[A][2 * j] = (_Float16)(p0 - (float)pr.x);
              pl[A][2 * j + 1] = (_Float16)(p1 - (float)pr.y);
            } else {
              l = __builtin_amdgcn_fdot2(pr, ones, l, false);   // the sum of what is multiplied
            }
          }
        const uint8_t* const v = vals + (i & 1) * HELD;
#pragma unroll
        for (int A = 0; A < 2; ++A)
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            const half8_t vc = __builtin_bit_cast(half8_t, lds16(v + ((A * TILES + t) * 64 + lane) * 16));
            acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vc, pf[A], acc[t], 0, 0, 0);
            if constexpr (FINE) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vc, pl[A], acc[t], 0, 0, 0);
          }
        spread_values(i + 1);
        spread_keys(i + 2);
        sc = next;
        ++i;
        if (i < blocks) pass = settle(i, hide, sc);
        if (far && !pass) settle_far();   // (in the outer loop otherwise)
      } while (i < blocks && !pass);
    }
  }

  const float sum = half_sum(l);
  const int r = w_r0 + (int)col, qi = r / a.ratio, hh = r - qi * a.ratio;
  if (r >= rows) return;
  if (!whole) {   // sums, and 2^base that they are held times
    const int64_t place = ((int64_t)blockIdx.x * a.parts + blockIdx.y) * ROWS + (r - r0);
    float* const to = a.acc + place * D;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int bb = 0; bb < 4; ++bb)
          *reinterpret_cast<f32x4*>(to + 64 * g + 4 * (8 * u + 4 * (int)half + bb)) =
              f32x4{acc[2 * g][4 * u + bb], acc[2 * g][8 + 4 * u + bb], acc[2 * g + 1][4 * u + bb],
                    acc[2 * g + 1][8 + 4 * u + bb]};
    if (half == 0) *reinterpret_cast<f32x2*>(a.ml + 2 * place) = f32x2{kTileShift - m, sum};
    return;
  }
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;   // 0: nothing seen; NaN stays
  const int64_t o = (int64_t)(sq.c0 + qi) * a.n_heads + head * a.ratio + hh;
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int bb = 0; bb < 4; ++bb) {
        const f32x4 v = {acc[2 * g][4 * u + bb], acc[2 * g][8 + 4 * u + bb], acc[2 * g + 1][4 * u + bb],
                         acc[2 * g + 1][8 + 4 * u + bb]};
        store4(a, o * D + 64 * g + 4 * (8 * u + 4 * (int)half + bb), v * inv);
      }
  if (a.lse && half == 0) a.lse[o] = (__builtin_amdgcn_logf(sum) + m - kTileShift) * kLn2;
}

// Joins the parts of the tiles that were cut: blockIdx.x is the tile as above, a
// thread takes four channels of a row. A launch of its own, since a tile's sums
// are up to 128 rows times 64 parts: one workgroup a tile would read for longer
// than the parts take.
template <int G>
__global__ __launch_bounds__(256) void k_kv4_attn_join(KvAttn a) {
  constexpr int D = 64 * G;
  const uint32_t bh_n = (uint32_t)(a.batch * a.cache.heads);
  const uint32_t bh = blockIdx.x % bh_n;
  const int b = (int)(bh / (uint32_t)a.cache.heads), head = (int)(bh % (uint32_t)a.cache.heads);
  Seq sq;
  if (!seq_from(a, a.cu[b], a.cu[b + 1], a.lens[b], sq)) return;
  const int rows = sq.nq * a.ratio, rts = (rows + kRowTile - 1) / kRowTile;
  const int rt = rts - 1 - (int)(blockIdx.x / bh_n);
  if (rt < 0) return;
  const int e = (int)(blockIdx.y * 256 + threadIdx.x), in_tile = e / (D / 4), c = e % (D / 4);
  const int r = rt * kRowTile + in_tile;
  if (r >= rows) return;
  const Reach re = tile_reach(a, sq, rows, rt * kRowTile);
  const int per = part_blocks(a, re), parts = (re.ns + re.nw + per - 1) / per;
  if (parts <= 1) return;
  const int64_t place = (int64_t)blockIdx.x * a.parts * kRowTile + in_tile;
  const float* const ml = a.ml + 2 * place;
  const float* const acc = a.acc + place * D + 4 * c;
  float low = -kNoMax;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) low = fminf(low, ml[p * (2 * kRowTile)]);
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const f32x2 x = *reinterpret_cast<const f32x2*>(ml + p * (2 * kRowTile));
    const float f = __builtin_amdgcn_exp2f(low - x.x);
    sum = __builtin_fmaf(x.y, f, sum);
    v += *reinterpret_cast<const f32x4*>(acc + (int64_t)p * (kRowTile * D)) * f;
  }
  const int qi = r / a.ratio, hh = r - qi * a.ratio;
  const int64_t o = (int64_t)(sq.c0 + qi) * a.n_heads + head * a.ratio + hh;
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;   // 0: nothing seen; NaN stays
  store4(a, o * D + 4 * c, v * inv);
  if (a.lse && c == 0) a.lse[o] = (__builtin_amdgcn_logf(sum) - low) * kLn2;
}

}  // namespace

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
