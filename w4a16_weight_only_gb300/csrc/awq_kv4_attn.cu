// Host side of awq_attention_kv4: how a call is cut, its workspace, and the choice of a kernel
// (awq_kv4_attn.cuh).
#include "awq_kv4_attn.cuh"

namespace awq {
namespace {

using namespace kv4;

int row_tile(const AttentionKv4Problem& p) {  // query rows of a unit, in eights
  const int64_t rows = static_cast<int64_t>(p.n) * (p.Hq / p.cache.heads);
  return rows > 8 && p.cache.head_dim <= 128 ? 2 : 1;
}

size_t part_bytes(const AttentionKv4Problem& p, int nt) { return static_cast<size_t>(8 * nt) * (p.cache.head_dim + 2) * 4; }

int most_blocks(const AttentionKv4Problem& p, int nt, int sms) { return sms * blocks_per_sm(p.cache.head_dim, nt); }

// A unit per block up to this many tiles (eight warps, 16 tiles each), where all units run at once.
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
