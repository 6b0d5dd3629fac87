// w4_parts.h - rows of the parts that the tile kernel of the 4-bit product works on (w4_tile.hip); plain C++, for the host too.
#pragma once

#ifdef __HIPCC__
#define MOE_W4_FN __host__ __device__ __forceinline__
#else
#define MOE_W4_FN inline
#endif

namespace moe {

constexpr int kW4PartRows = 128;

// A group's tile of up to `tile_rows` rows, of which part `part` is rows 128 part .. of the tile: how many it has, where the
// group has `left` rows from the tile's first one on. The rest of a longer group belongs to its next tile.
MOE_W4_FN int w4_part_rows(int left, int tile_rows, int part) {
    const int in_tile = (left < tile_rows ? left : tile_rows) - part * kW4PartRows;
    return in_tile < 0 ? 0 : in_tile < kW4PartRows ? in_tile : kW4PartRows;
}

}  // namespace moe
