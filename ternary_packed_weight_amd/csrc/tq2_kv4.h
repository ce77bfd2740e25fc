// The 4-bit key/value cache: its layout, and the launch interface between the
// C ABI (tq2_kv4_api.cpp) and the gfx950 kernels (tq2_kv4.hip).  Not part of
// the public ABI.
//
// One (page, head) block holds P tokens: [key codes P*D/2][value codes P*D/2]
// [key (s, z) pairs P*4][value (s, z) pairs P*4] bytes.  Key codes are token
// major, so a lane's 16-byte load is 32 consecutive channels of one token:
// the operand rows of K Q^T.  P V contracts over tokens, so its operand needs
// eight tokens of one channel in a lane: value codes stand in tiles of 32
// tokens, [tile][token/8][channel/4][token%8] 16-bit units of four channels,
// and a wave's load of a tile is linear.
#pragma once
#include <stddef.h>
#include <stdint.h>

#if defined(__HIPCC__)
#define TQ2_HD __host__ __device__ inline
#else
#define TQ2_HD inline
#endif

namespace tq2 {

constexpr int kKvTile = 32;  // tokens of a value tile, and of one attention step

TQ2_HD int64_t kv4_block_bytes(int P, int D) { return (int64_t)P * (D + 8); }
// Byte offsets inside a (page, head) block, for token t of the page.
TQ2_HD int64_t kv4_key_at(int D, int t) { return (int64_t)t * (D / 2); }
TQ2_HD int64_t kv4_value_unit_at(int P, int D, int t, int unit) {
  return (int64_t)P * (D / 2) + (int64_t)(t / 32) * (16 * D) +
         ((((t % 32) / 8) * (D / 4) + unit) * 8 + t % 8) * 2;
}
TQ2_HD int64_t kv4_key_pair_at(int P, int D, int t) { return (int64_t)P * D + t * 4; }
TQ2_HD int64_t kv4_value_pair_at(int P, int D, int t) { return (int64_t)P * (D + 4) + t * 4; }
// The block of a slot's token for one head, or -1 where the slot names no page.
TQ2_HD int64_t kv4_slot_block(int64_t slot, int64_t pages, int Hk, int P, int D, int head, int* t) {
  if (slot < 0 || slot / P >= pages) return -1;
  *t = (int)(slot % P);
  return ((slot / P) * Hk + head) * kv4_block_bytes(P, D);
}
// Whether a table's entry names a page: one unsigned comparison, as a negative
// entry is past any limit.
TQ2_HD uint32_t kv4_page_limit(int64_t pages) { return pages < INT32_MAX ? (uint32_t)pages : (uint32_t)INT32_MAX + 1u; }
TQ2_HD bool kv4_page_there(int32_t page, uint32_t limit) { return (uint32_t)page < limit; }
// The block of a page that a table names, or -1 where it names none (the
// layout's definition for host tests; the kernels step through blocks by units
// of 16 bytes).
TQ2_HD int64_t kv4_page_block(int32_t page, int64_t pages, int Hk, int P, int D, int head) {
  if (!kv4_page_there(page, kv4_page_limit(pages))) return -1;
  return ((int64_t)page * Hk + head) * kv4_block_bytes(P, D);
}

// The part of a sequence that a tile of rows reads, cut into at most nsplit
// splits of whole steps (the kernels ask for one: they deal by length, below).
// Rows are (new token, query head of the key head); n new tokens, c cached
// tokens.
struct Kv4Range {
  int first, last;  // tiles of 32 tokens, [first, last)
  int chunk;        // tiles of one split
  int splits;       // splits that hold any (0: no row sees a token)
};
// Tiles of a part, such that `parts` parts of whole steps hold all of them.
TQ2_HD int kv4_chunk(int tiles, int parts, int step) { return ((tiles + parts - 1) / parts + step - 1) / step * step; }
// Part `part` of the tiles, [first, last); the last ones may be empty.
struct Kv4Part {
  int first, last;
};
TQ2_HD Kv4Part kv4_part(int tiles, int parts, int part, int step) {
  const int chunk = kv4_chunk(tiles, parts, step), first = chunk * part;
  return {first < tiles ? first : tiles, first + chunk < tiles ? first + chunk : tiles};
}
TQ2_HD Kv4Range kv4_range(int n, int c, int G, int row0, int rows, int window, int nsplit, int waves) {
  const int i0 = row0 / G;
  int i1 = (row0 + rows - 1) / G;
  if (i1 > n - 1) i1 = n - 1;
  int64_t end = (int64_t)c - n + i1 + 1, begin = window > 0 ? (int64_t)c - n + i0 + 1 - window : 0;
  if (end > c) end = c;
  if (begin < 0) begin = 0;
  Kv4Range r{0, 0, 1, 0};
  if (end <= begin) return r;
  r.first = (int)(begin / kKvTile);
  r.last = (int)((end + kKvTile - 1) / kKvTile);
  const int tiles = r.last - r.first;
  r.chunk = kv4_chunk(tiles, nsplit, waves);
  r.splits = (tiles + r.chunk - 1) / r.chunk;
  return r;
}
TQ2_HD int kv4_clamp(int64_t v, int64_t lo, int64_t hi) { return (int)(v < lo ? lo : v > hi ? hi : v); }

// New tokens [q0, q0 + n) and cached tokens c of a sequence, held inside the
// call's own sizes whatever the arrays on the device say: rows s0 .. s1 of T,
// at most max_q of them, ctx of at most `most` cached tokens.
struct Kv4Seq {
  int64_t q0;
  int n, c;
};
TQ2_HD Kv4Seq kv4_seq(int64_t s0, int64_t s1, int32_t ctx, int64_t T, int max_q, int64_t most) {
  Kv4Seq q;
  q.q0 = s0 < 0 ? 0 : s0 > T ? T : s0;
  q.n = kv4_clamp((s1 > T ? T : s1) - q.q0, 0, max_q);
  q.c = kv4_clamp(ctx, 0, most);
  return q;
}

// Workgroups are dealt to the rows' tokens by length.  An
// entry is a tile of `rows` rows of a sequence; it has tiles of 32 tokens to
// read for every key head (one where its rows see no token, so that their
// zeros are written; none where it has no row), in units of 2^grain tiles.
TQ2_HD int kv4_tiles(const Kv4Seq& q, int G, int row0, int rows, int window, int* first) {
  const Kv4Range r = kv4_range(q.n, q.c, G, row0, rows, window, 1, 1);
  *first = r.first;
  if (row0 >= (int64_t)q.n * G) return 0;
  return r.last > r.first ? r.last - r.first : 1;
}
TQ2_HD uint32_t kv4_units(int tiles, int grain) { return (uint32_t)(((int64_t)tiles + (1 << grain) - 1) >> grain); }
// Units of one workgroup at most, such that all entries take `budget`
// workgroups and one more for each (entry, head) at most.  The units of all
// heads are below 2^31 and one for each (that is what the grain is for).
TQ2_HD uint32_t kv4_share(uint32_t units, int Hk, uint32_t budget, uint32_t least) {
  const uint32_t s = (units * (uint32_t)Hk + budget - 1) / budget;
  return s < least ? least : s;
}
// What an entry takes: workgroups, slots for the parts of its split heads, heads that are split.
struct Kv4Take {
  uint32_t wgs, slots, splits;
};
TQ2_HD Kv4Take kv4_take(uint32_t units, int Hk, uint32_t share) {
  const uint32_t n = (units + share - 1) / share;
  return {n * Hk, n > 1 ? n * Hk : 0, n > 1 ? (uint32_t)Hk : 0};
}

// What a workgroup does: part `part` of `parts` of an (entry, head), its slot,
// and its group where the parts are joined.
struct Kv4Work {
  int32_t e, head, parts, part, slot, group, pad[2];
};
// A split row tile: its sequence's first row of q and out, its own first row
// and the rows of the sequence, and the slots of its parts.  The first group's
// `groups` says how many there are; count < 2: nothing to join.
struct Kv4Group {
  int32_t q0, row0, rows, head, slot, count, groups, pad;
};
// What a call launches: row tiles of 16 a wave (mt), whether the waves of a
// workgroup share rows and split tokens (few rows) or the other way round.
struct Kv4AttnPlan {
  int mt, tiles, budget, least, grain, groups, slots, rows;
  int64_t grid;
  bool few, list;
  size_t ws_bytes;
};
constexpr int kWaves = 4;  // of a workgroup
// Workgroups of the kernel for few rows that are resident on a CU, by its registers.
TQ2_HD constexpr int few_resident(int D, int MT) { return D * MT > 256 ? 1 : 2; }
TQ2_HD Kv4AttnPlan plan_kv4_attn(int Hq, int Hk, int D, int P, int width, int B, int max_q, int window) {
  Kv4AttnPlan p{};
  const int64_t rows = (int64_t)max_q * (Hq / Hk);
  // the most tiles that a row tile can see: the table's, or a window's where those are fewer
  const int64_t held = (int64_t)width * P / kKvTile, seen = ((int64_t)window + max_q + 31) / kKvTile + 1;
  const int64_t tiles = window > 0 && seen < held ? seen : held;
  // Split tokens (few) or rows (many)?  Few workgroups or short texts are a
  // matter of latency, where the waves that split tokens win even if rows are
  // many.  Measured (us, few and many; sequences, new tokens, cached tokens),
  // heads of 128, 2 key heads of 16 query heads: 1, 24, 8000 27 and 44; 2, 64,
  // 8000 52 and 64; 4, 64, 300 13 and 19; 1, 512, 512 18 and 24; 1, 160, 6000
  // 58 and 61; but 8, 24, 8000 89 and 70; 1, 200, 20000 180 and 122.  8 key
  // heads of 4: 1, 24, 8000 27 and 57; 1, 512, 1000 31 and 39; 8, 24, 8000 85
  // and 84; 1, 200, 20000 171 and 133.  Heads of 64: the same order, 1, 24,
  // 8000 22 and 39, 8, 24, 8000 73 and 58.  Where it holds less: near the last
  // bound with thousands of rows of short text (4, 200, 1000 56 and 39; 1, 1000,
  // 1000 47 and 39), and for heads of 256 (1, 512, 512 38 and 28; 8, 12, 8000 85
  // and 78; 1, 24, 8000 38 and 57).  64 rows of very many sequences lose 10 %
  // with few (64, 4, 8000 93 and 83): what few keeps of a probability is worth
  // more there.  (By the table's width: a window must not ask for more
  // workspace than the call without one.)
  const int64_t all = (int64_t)B * Hk * rows;
  p.few = rows <= 64 || all <= 4096 || all * held <= 1 << 20;
  p.mt = p.few ? (rows > 16 ? 2 : 1) : D < 256 && rows > 256 ? 2 : 1;
  p.rows = (p.few ? 16 : 64) * p.mt;
  p.tiles = (int)((rows + p.rows - 1) / p.rows);
  const int64_t items = (int64_t)B * p.tiles * Hk;
  p.grid = items;
  // Tiles that a part has at least, and that a row tile has at least to be
  // dealt.  Few rows: two tiles a wave cost what the join does (drafts: 16
  // 15.9 us, 8 17.9, 32 19.2).  Many: the list and the join take 15 us, eleven
  // tiles' time, which pays early where there are few workgroups: 64 of 63
  // tiles take 48 us in parts of 8 or more and 67 undealt, 128 of 100 68 and 78
  // in parts of 48, but 226 of 63 75 and 67 undealt, of 100 100 and 90 in parts
  // of 48 (heads of 128; of 64 alike).
  const bool lone = items < 192;
  p.least = p.few ? 4 * kWaves : lone ? 8 : 48;
  if (tiles > (p.few ? p.least : lone ? 32 : 96)) {
    // as many workgroups as are resident at once, a few less where parts of 64
    // KiB would pass 64 MiB.  Many row tiles need them too (5120 of up to 125
    // tiles 389 us, with 128 workgroups 450, undealt 505; 16384 1034, 1095 and
    // 1189), until their list takes the memory.
    p.budget = p.few ? 256 * few_resident(D, p.mt) : items <= 1 << 15 ? 490 : 128;
    while (items * tiles >> p.grain > INT32_MAX) ++p.grain;
    p.grid += p.budget;
    // up to two lengths a lane; 256 sequences take as long either way, 1024 459 us without a list and 251 with one
    p.list = !p.few || (int64_t)B * p.tiles > 128;
    p.slots = 2 * p.budget;
    p.groups = (int)(items < p.budget ? items : p.budget);
  }
  p.ws_bytes = p.groups ? (size_t)p.slots * p.rows * (D + 2) * 4 + (size_t)p.groups * sizeof(Kv4Group) +
                              (p.list ? (size_t)p.grid * sizeof(Kv4Work) : 0)
                        : 0;
  return p;
}

}  // namespace tq2

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
namespace tq2 {

enum { kF16 = 0, kBF16 = 1, kF32 = 2 };  // TQ2_DTYPE_*

struct RopeArgs {
  const void *q, *k;
  void *q_out, *k_out;
  const float *q_weight, *k_weight, *inv_freq;
  const int32_t* positions;
  int64_t q_ts, q_hs, k_ts, k_hs, T;  // strides in elements
  int32_t Hq, Hk, D, rot, interleaved;
  float eps;
};
hipError_t launch_qk_norm_rope(const RopeArgs& a, int in_dtype, int out_dtype, hipStream_t s);

struct Kv4StoreArgs {
  const void *k, *v;
  uint8_t* cache;
  const int64_t* slots;
  int64_t k_ts, k_hs, v_ts, v_hs, T, pages;
  int32_t Hk, D, P;
};
hipError_t launch_kv4_store(const Kv4StoreArgs& a, int dtype, hipStream_t s);

struct Kv4LoadArgs {
  const uint8_t* cache;
  const int64_t* slots;
  void *k, *v;  // [T][Hk][D]; either may be null
  int64_t T, pages;
  int32_t Hk, D, P;
};
hipError_t launch_kv4_load(const Kv4LoadArgs& a, int dtype, hipStream_t s);

struct Kv4AttnArgs {
  const void* q;
  void* out;
  float* lse;
  const uint8_t* cache;
  const int32_t *table, *ctx, *q_start;
  // Parts of split rows: [slots][rows of a workgroup][D] sums, then
  // [slots][rows][2] (reference, weight), then the groups to join.
  float* part;
  int64_t q_ts, q_hs, table_stride, T, pages;
  int32_t B, max_q, width, Hq, Hk, G, D, P, window;
  int32_t tiles;   // row tiles of a sequence
  int32_t budget;  // workgroups to deal by length; 0: each (entry, head) is one's
  int32_t least, grain;
  int32_t list;    // whether the work stands in a list
  int32_t slots, rows, groups;
  float scale;
};
hipError_t launch_kv4_attn(Kv4AttnArgs a, const Kv4AttnPlan& p, int dtype, hipStream_t s);

}  // namespace tq2
#endif
