// Host-side planning of an fp8-cache decode: the widened bf16 copy's place in
// the workspace and the groups of sequences a call runs in.  Shared by api.cu
// and the host checker in tests/partition_check.cu.
#pragma once

#include <stddef.h>

#include "common.cuh"

namespace mla {

// The fp8 cache's widened bf16 copy, placed after the split-KV workspace:
// a scratch block table int32 [B * max_blocks] and a dense bf16 cache
// [B * max_blocks, 64, 576] (block b * max_blocks + j holds logical block j
// of sequence b).  Its block ids and TMA row coordinates must fit int32.
constexpr long long kMaxWideBlocks = 1LL << 24;

struct WideLayout {
  size_t table, cache, total;
};

inline WideLayout wide_layout(size_t split_ws_total, int B, int max_blocks) {
  const size_t n = size_t(B) * size_t(max_blocks);
  WideLayout w;
  w.table = align256(split_ws_total);
  w.cache = align256(w.table + n * 4);
  w.total = w.cache + n * kBlock * kRow * 2;
  return w;
}

// Bytes one group of `B` sequences on `P` engines needs: its split-KV
// scratch followed by its widened copy (0 when the copy's block count is out
// of range).
inline size_t fp8_group_bytes(int B, int rows, int max_blocks, int P) {
  if (static_cast<long long>(B) * max_blocks > kMaxWideBlocks) return 0;
  return wide_layout(ws_layout(B, rows, P).total, B, max_blocks).total;
}

// Groups of consecutive sequences, Bg per group (the last one may be short)
// on at most Pg engines, such that every group fits `ws_bytes`: the whole
// batch on P engines when it fits; else fewer engines first (halving), then
// smaller groups (halving, engines back at engines_for(group size)).  Bg = 0
// when not even one sequence on one engine fits.  A group of n sequences runs
// on min(Pg, engines_for(n)) engines.
struct Fp8Plan {
  int Bg, Pg;
};

template <class EnginesFor>
inline Fp8Plan plan_fp8_groups(int B, int rows, int max_blocks, int P, size_t ws_bytes, EnginesFor engines_for) {
  int Bg = B, Pg = P;
  for (;;) {
    const size_t need = fp8_group_bytes(Bg, rows, max_blocks, Pg);
    if (need != 0 && need <= ws_bytes) return Fp8Plan{Bg, Pg};
    if (Pg > 1) {
      Pg = (Pg + 1) / 2;
    } else if (Bg > 1) {
      Bg = (Bg + 1) / 2;
      Pg = engines_for(Bg);
      if (Pg < 1) Pg = 1;
    } else {
      return Fp8Plan{0, 0};
    }
  }
}

// A chunk call's tile: query rows that one engine attends at once, whole
// tokens of one sequence.
constexpr int kChunkTileRows = 256;

// Workspace of a chunk call of T tokens, B sequences and H heads on P engines:
// error word; tile count; tile list; fp32 pieces of cut tiles (at most two per
// engine).  A sequence of n tokens has ceil(n / (256 / H)) tiles.
struct ChunkLayout {
  int max_tiles;
  size_t n_tiles, tile_off, tiles, pre, engines, lse_part, o_part, total;
};

inline ChunkLayout chunk_layout(int T, int B, int H, int P) {
  ChunkLayout w;
  w.max_tiles = T / (kChunkTileRows / H) + B;
  w.n_tiles = 256;
  w.tile_off = 512;
  w.tiles = align256(w.tile_off + (size_t(B) + 1) * 4);
  w.pre = align256(w.tiles + size_t(w.max_tiles) * 16);
  w.engines = align256(w.pre + (size_t(w.max_tiles) + 1) * 8);
  w.lse_part = align256(w.engines + size_t(P) * 64);
  w.o_part = align256(w.lse_part + size_t(2 * P) * kChunkTileRows * 4);
  w.total = align256(w.o_part + size_t(2 * P) * kChunkTileRows * kDc * 4);
  return w;
}

// Workspace of an eviction: error word, moves per sequence, move lists (at
// most half of a sequence's slots are free below its budget and filled from
// behind it).
constexpr int kMaxEvictBlocks = 65536;  // table width: two bits per slot stay in one cluster's shared memory

struct EvictLayout {
  size_t n_moves, moves, total;
};

inline EvictLayout evict_layout(int B, int max_blocks) {
  EvictLayout w;
  w.n_moves = 256;
  w.moves = align256(w.n_moves + size_t(B) * 4);
  w.total = w.moves + size_t(B) * max_blocks * (kBlock / 2) * 8;
  return w;
}

}  // namespace mla
