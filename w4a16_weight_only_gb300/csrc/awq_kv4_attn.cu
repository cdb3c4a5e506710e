// Host side of awq_attention_kv4: how a call is cut, its workspace, and the choice of a kernel
// (awq_kv4_attn.cuh).
#include "awq_kv4_attn.cuh"

namespace awq {
namespace {

using namespace kv4;

// Query rows of a unit, in eights.  Heads of 128, groups of 128, bf16, 32 sequences over up to 4096, by eight and by
// sixteen rows: 9 rows of a head 37 and 36 us, 16 37 and 36, 24 48 and 51, 32 58 and 52, 48 77 and 67; 4 over 2048, any of
// these, 19 and 23.  Heads of 64: 16 rows 30 and 31, 24 37 and 44, 32 44 and 44, 48 57 and 57.  (Three tiles of eight would
// serve 17 to 24 rows better.)  Heads of 256 have no registers for sixteen.
int row_tile(const AttentionKv4Problem& p) {
  const int64_t rows = static_cast<int64_t>(p.n) * (p.Hq / p.cache.heads);
  return rows > 8 && p.cache.head_dim <= 128 ? 2 : 1;
}

size_t part_bytes(const AttentionKv4Problem& p, int nt) { return static_cast<size_t>(8 * nt) * (p.cache.head_dim + 2) * 4; }

int most_blocks(const AttentionKv4Problem& p, int nt, int sms) { return sms * blocks_per_sm(p.cache.head_dim, nt); }

// A unit per block up to this many tiles (eight warps, 16 tiles each), where all units run at once.  Heads of 128, a unit
// per block and by the line: 8 units of 256 keys 9 and 13 us, of 1024 13 and 14, of 2048 19 and 16; 96 units of 700 12 and
// 19, of 2048 19 and 21; 296 units of 700 15 and 22, of 2048 26 and 31.
constexpr int kAlignedTiles = 128;

struct Layout {
  size_t firsts, line, bytes;  // parts first
};

Layout layout(const AttentionKv4Problem& p, int sms) {
  const int nt = row_tile(p), grid = most_blocks(p, nt, sms);
  Layout l;
  l.firsts = 2 * grid * part_bytes(p, nt);
  l.line = l.firsts + static_cast<size_t>(grid) * kWarps * part_bytes(p, nt);
  l.bytes = l.line + (static_cast<size_t>(p.B) + 2) * 8;
  return l;
}

}  // namespace

size_t attention_kv4_workspace_bytes(const AttentionKv4Problem& p, int sms) { return layout(p, sms).bytes; }

cudaError_t launch_attention_kv4(const AttentionKv4Problem& p, int sms) {
  Args a{};
  a.p = p;
  const cudaError_t e = status_word_ptr(&a.status);
  if (e != cudaSuccess) return e;
  const int nt = row_tile(p);
  a.group = p.Hq / p.cache.heads;
  a.row_tiles = static_cast<int>((static_cast<int64_t>(p.n) * a.group + 8 * nt - 1) / (8 * nt));
  a.tiles_per_page = p.cache.page_size / kTileKeys;
  const Layout l = layout(p, sms);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  a.parts = reinterpret_cast<float*>(ws);
  a.firsts = reinterpret_cast<float*>(ws + l.firsts);
  a.line = reinterpret_cast<int64_t*>(ws + l.line);
  // tiles of a sequence that its table and window allow, below 2^27, and units, below 2^32 (B n Hq < 2^31)
  int64_t tiles = static_cast<int64_t>(p.W) * a.tiles_per_page;
  if (p.window > 0) {
    const int64_t seen = (static_cast<int64_t>(p.window) + p.n + p.sinks) / kTileKeys + 3;
    if (seen < tiles) tiles = seen;
  }
  const int64_t units = static_cast<int64_t>(p.B) * p.cache.heads * a.row_tiles;
  const int most = most_blocks(p, nt, sms);
  a.aligned = tiles <= kAlignedTiles && units <= most;
  const int64_t need = a.aligned ? units : units * tiles / kWarps + 1;
  const int grid = static_cast<int>(need < most ? need : most);
  switch (p.cache.head_dim) {
    case 64: return run_64(a, nt, grid);
    case 96: return run_96(a, nt, grid);
    case 128: return run_128(a, nt, grid);
    default: return run_256(a, nt, grid);
  }
}

}  // namespace awq
