// Layout of a tile of the 4-bit cache: 16 tokens of one key/value head, 18 d bytes (include/attn_kv.h).
#pragma once

#include <cstdint>

namespace ea {

template <int D>
struct Kv4Tile {
  static constexpr int kPlaneDims = D < 128 ? D : 128;
  static constexpr int kPlanes = D / kPlaneDims;
  static constexpr int kGroups = kPlaneDims / 64;      // scale groups in a plane
  static constexpr int kRowBytes = kPlaneDims / 2;     // codes of one token in a plane
  static constexpr int kPlaneBytes = 16 * kRowBytes;
  static constexpr int kVOff = 8 * D;
  static constexpr int kKszOff = 16 * D;
  static constexpr int kVszOff = 17 * D;
  static constexpr int kBytes = 18 * D;
  static constexpr int kSzRow = D / 16;                // bytes of the (s, z) pairs of one token
};

// First byte of the tile that holds slot `slot` of head h, and the slot's row in it.
template <int D>
__device__ __forceinline__ long long kv4_tile_offset(int block, int off, int page, int Hk, int h) {
  return ((static_cast<long long>(block) * Hk + h) * (page >> 4) + (off >> 4)) * Kv4Tile<D>::kBytes;
}

}  // namespace ea
