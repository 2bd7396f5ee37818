// Rows (tokens x the heads that share a key/value head) of a sequence of the 8-bit cache's attention and their tiles: up to
// 2^31 - 1 rows, so that nothing may be added to a row's number that goes beyond them.
#pragma once

#include "plan.h"

namespace moe {

// Tiles of `tile` rows.
MOE_HD int kv8_tiles(int rows, int tile) { return rows > 0 ? (rows - 1) / tile + 1 : 0; }
// Rows from row0 on, of a tile of `tile`.
MOE_HD int kv8_rows_left(int rows, int row0, int tile) { return rows - row0 < tile ? rows - row0 : tile; }

}  // namespace moe
