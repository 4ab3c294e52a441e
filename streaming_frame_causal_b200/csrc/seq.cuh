// seq.cuh -- what the per-sequence decode kernels share: their parameters, and the
// division of the work.
//
// Every sequence b has its own position pos[b] (in device memory, so that a
// captured step can be replayed as the positions advance) and so its own number
// of keys.  An item is one (sequence, KV head, group of up to 8 of its query
// heads); its keys are cut into tiles of 128.  The tiles of all items, in order
// (sequence, KV head, group), form one line of T tiles, and CTA c of G takes the
// tiles [c T / G, (c + 1) T / G): the shares differ by one tile at most, whatever
// the lengths.  A CTA that holds an item whole writes its output; an item cut
// between CTAs leaves partial results, two slots per CTA at most (the item that
// runs into its share, and the one that runs out of it), which a second kernel
// merges in the order of the tiles.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "ptx.cuh"
#include "tile_sched.h"

namespace swa {

constexpr int kSeqKeys = 128;     // keys of a tile
constexpr int kSeqRows = 8;       // query heads of an item
constexpr int kSeqMaxCtas = 512;  // CTAs that the workspace has partial slots for
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
  int* cum;               // [B + 1] tiles of an item of each sequence, summed
  int4* share;            // [ctas] {sequence, item of it, first tile, tiles}
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
  int ctas;
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

// CTAs that share a line of T tiles: no share is empty, so that the pieces of a cut
// item are those of consecutive CTAs
SWA_DEV int seq_ctas(const SeqParams& p, int64_t T) { return T < p.ctas ? static_cast<int>(T) : p.ctas; }

// CTA that owns tile t of the line of T: the c with c T / G <= t < (c + 1) T / G
SWA_DEV int seq_owner(int64_t t, int64_t T, int ctas) { return static_cast<int>(((t + 1) * ctas - 1) / T); }

// A run of tiles of one item within a CTA's share.
struct SeqRun {
  int b, item, t0, tiles;  // tiles [t0, t0 + tiles) of the item
  int of;                  // tiles that the item has
  int slot;                // partial slot; -1: the item is whole, its output is written
};

// Walks a CTA's share.  Every role of a CTA walks it for itself.
struct SeqWalk {
  int b, item, t0, left, of;
  SWA_DEV void start(const SeqParams& p, int cta) {
    const int4 s = p.share[cta];
    b = s.x;
    item = s.y;
    t0 = s.z;
    left = s.w;
    of = left > 0 ? seq_tiles(p, b) : 0;
  }
  SWA_DEV bool next(const SeqParams& p, int cta, SeqRun& r) {
    if (left <= 0) return false;
    while (item >= p.items || of == 0) {  // on to the next sequence that has keys
      item = 0;
      ++b;
      if (b >= p.B) return false;
      of = seq_tiles(p, b);
    }
    r.b = b;
    r.item = item;
    r.t0 = t0;
    r.of = of;
    r.tiles = min(left, of - t0);
    const bool whole = r.tiles == of;
    // with a shared prefix every item is merged with the prefix's pieces
    r.slot = whole ? (p.N > 0 ? 2 * p.ctas + b * p.items + item : -1) : 2 * cta + (t0 == 0 ? 1 : 0);
    left -= r.tiles;
    t0 = 0;
    ++item;
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
int seq_tc_ctas(int D, bool kv8, int sms);
cudaError_t launch_seq_tc(const SeqParams& p, int D, bool kv8, cudaStream_t stream);

}  // namespace swa
