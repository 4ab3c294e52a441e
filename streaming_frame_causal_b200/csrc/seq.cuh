// seq.cuh -- what the per-sequence decode kernels share: their parameters, and the
// division of the work.
//
// Every sequence b has its own position pos[b] (in device memory, so that a
// captured step can be replayed as the positions advance) and so its own number
// of keys, cut into tiles of 128.  An item is one (sequence, KV head, group of up to 8
// of its query heads).  The tiles of all sequences, in order, form one line of T, and
// team c of C takes the tiles [c T / C, (c + 1) T / C): the shares differ by one tile at
// most, whatever the lengths.  A team is one CTA per item of a sequence, and its
// CTAs walk the same tiles side by side: a token's KV heads lie next to one another
// in a cache, so the team reads whole rows of memory together.  (Shares of a line of
// the items' tiles, with the heads' CTAs at different places, ran the 8-bit decode of 64
// x 4096 tokens x 8 heads in 128 us against 97.)  A CTA that holds an item whole
// writes its output; an item cut between teams leaves partial results, two slots
// per CTA at most (the sequence that runs into its share, and the one that runs out of
// it), which a second kernel merges in the order of the tiles.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "ptx.cuh"
#include "tile_sched.h"

namespace swa {

constexpr int kSeqKeys = 128;     // keys of a tile
constexpr int kSeqRows = 8;       // query heads of an item
constexpr int kSeqMaxCtas = 640;  // CTAs that the workspace has partial slots for (or one team, if that is more)
constexpr int kSeqCols = 16;      // query columns of the tensor-core products
constexpr int kSeqMaxSplits = 64; // pieces of a shared prefix

struct SeqParams {
  const void* q;          // [B, Hq, D]
  const void* k_new;      // [B, Hkv, D]
  const void* v_new;
  void* k_cache;          // [B, W, Hkv, D]
  void* v_cache;
  uint8_t* k_exp;         // 8-bit caches: [B, Hkv, W]
  uint8_t* v_exp;
  const long long* pos;   // [B]
  void* out;              // [B, Hq, D]
  int* selected;          // block-sparse: [B, Hkv, n_select] ascending, -1 behind
  void* bounds;           // [B, Hkv, blocks, 2, D]
  uint64_t* score;        // [B * Hkv, blocks] sortable
  const void* k_prefix;   // [N, Hkv, D]
  const void* v_prefix;
  int* cum;               // [B + 1] tiles of the sequences, summed
  int4* share;            // [teams] {sequence, first tile of it, tiles}
  float* part_o;          // [slots, 8, D]
  float* part_ml;         // [slots, 8, 2] maximum in log2 units, sum
  float* pre_o;           // [splits, B * Hq, D]
  float* pre_ml;          // [splits, B * Hq, 2]
  uint8_t* q8;            // 8-bit caches: [B * Hkv, 16, D] the queries as two e4m3 terms
  float* q_scale;         // [B * Hq] 2^e of each
  int* err;
  int W, B, Hq, Hkv, G;   // G query heads per KV head
  int groups, items;      // groups of 8 heads per KV head; items per sequence = Hkv * groups
  int block, n_select, n_first, n_last, n_blocks;  // block-sparse (block = 0: all keys)
  int N, splits;          // shared prefix
  int teams, ctas;        // ctas = teams * items
  int merge_warps;        // warps that merge one row's pieces
  float scale_log2;
};

// tokens of sequence b in the cache, the new one included (0: an idle row)
SWA_DEV int seq_tokens(const SeqParams& p, int b) {
  const long long pos = p.pos[b];
  return pos < 0 ? 0 : (pos >= p.W - 1 ? p.W : static_cast<int>(pos) + 1);
}

// tiles of each item of sequence b
SWA_DEV int seq_tiles(const SeqParams& p, int b) {
  const int n = seq_tokens(p, b);
  if (p.block == 0) return (n + kSeqKeys - 1) / kSeqKeys;
  const int blocks = min((n + p.block - 1) / p.block, p.n_select);
  return (blocks * p.block + kSeqKeys - 1) / kSeqKeys;
}

// teams that share a line of T tiles: no share is empty, so that the pieces of a cut
// item are those of consecutive teams
SWA_DEV int seq_teams(const SeqParams& p, int T) { return T < p.teams ? T : p.teams; }

// team that owns tile t of the line of T: the c with c T / C <= t < (c + 1) T / C
SWA_DEV int seq_owner(int t, int T, int teams) {
  return static_cast<int>((static_cast<int64_t>(t + 1) * teams - 1) / T);
}

// A run of tiles of one sequence within a CTA's share.
struct SeqRun {
  int b, t0, tiles;  // tiles [t0, t0 + tiles) of the CTA's item of sequence b
  int slot;          // partial slot; -1: the item is whole, its output is written
};

// Walks a CTA's share.  Every role of a CTA walks it for itself.
struct SeqWalk {
  int cta, item, b, t0, left, of;
  SWA_DEV void start(const SeqParams& p, int c) {
    cta = c;
    item = c % p.items;
    const int4 s = p.share[c / p.items];
    b = s.x;
    t0 = s.y;
    left = s.z;
    of = left > 0 ? seq_tiles(p, b) : 0;
  }
  SWA_DEV bool next(const SeqParams& p, SeqRun& r) {
    if (left <= 0) return false;
    while (t0 >= of) {  // on to the next sequence that has keys
      if (++b >= p.B) return false;
      t0 = 0;
      of = seq_tiles(p, b);
    }
    r.b = b;
    r.t0 = t0;
    r.tiles = min(left, of - t0);
    // with a shared prefix every item is merged with the prefix's pieces
    r.slot = r.tiles == of ? (p.N > 0 ? 2 * p.ctas + b * p.items + item : -1) : 2 * cta + (t0 == 0 ? 1 : 0);
    left -= r.tiles;
    t0 = of;
    return true;
  }
};

// Key r of tile t of an item: its slot in the cache, or -1 behind the item's keys.
SWA_DEV int seq_slot(const SeqParams& p, int b, int kvh, int n_tokens, int t, int r) {
  const int i = t * kSeqKeys + r;
  if (p.block == 0) return i < n_tokens ? i : -1;
  const int j = i / p.block;
  if (j >= p.n_select) return -1;
  const int blk = p.selected[(static_cast<int64_t>(b) * p.Hkv + kvh) * p.n_select + j];
  const int slot = blk * p.block + (i - j * p.block);
  return (blk >= 0 && slot < n_tokens) ? slot : -1;
}

// columns that G query heads take: 1, 2, 4 or 8
SWA_HD int seq_head_columns(int G) { return G <= 2 ? G : (G <= 4 ? 4 : 8); }

// the tensor-core kernel (seq_tc.cu), behind the preparation on the same stream: 16-bit
// queries, head_dim 64 or 128, at most 8 query heads per KV head; p.ctas = seq_tc_ctas
int seq_tc_ctas(int D, int G, bool kv8, int sms);
cudaError_t launch_seq_tc(const SeqParams& p, int D, bool kv8, cudaStream_t stream);

}  // namespace swa
