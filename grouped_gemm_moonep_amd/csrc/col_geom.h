// Where the loads of a column tile read: an operand stored [k][n], n contiguous,
// 64 k rows of one or two regions of columns.  Plain integer arithmetic, so that
// a host program can enumerate it.
#pragma once

#include <stdint.h>

namespace moonep {

// Marks an offset as out of range: added to any valid offset it stays past num_records (at most
// 2^31 - 1), where a load reads 0.
constexpr uint32_t kOob = 0x80000000u;

// COLS columns of a region, loaded by WAVES waves: every load of a wave takes kRows whole rows, 16
// bytes a lane.
template <int COLS, int WAVES>
struct ColGeom {
  static constexpr int kLanes = COLS / 8;                    // of a row
  static constexpr int kRows = 64 / kLanes;                  // of a load
  static constexpr int kLoads = 64 / (WAVES * kRows);        // of a wave
  static constexpr int kRegion = 64 * COLS * 2;              // bytes in LDS
  // 16-byte chunk c of row k sits at c ^ swz(k): the rows that a transposing read takes together lie
  // on distinct banks (four of 256 bytes; of 128 bytes two in each 256-byte window of the LDS).
  static constexpr int swz(int k) { return 4 * (COLS == 128 ? k & 3 : (k >> 1) & 1); }
  // Bytes from a region's first element to the end of its last row's valid columns: no byte past
  // the matrix is in range, whatever the offset.  A matrix has fewer than 2^31 bytes.
  static constexpr uint32_t bytes(uint32_t ld2, int k_total, int nv) {
    return k_total > 0 && nv > 0 ? (uint32_t)(k_total - 1) * ld2 + (uint32_t)(2 * nv) : 0;
  }
  // A lane's first load of k-block 0 (w: the wave's number within the tile), or the mark past the
  // region's nv valid columns.
  static constexpr uint32_t lane(int w, int lane, uint32_t ld2, int nv) {
    const int k = 64 / WAVES * (w % WAVES) + lane / kLanes;  // load i adds kRows i rows
    const int col = 8 * ((lane % kLanes) ^ swz(k));
    return col < nv ? (uint32_t)k * ld2 + (uint32_t)(col * 2) : kOob;
  }
  // Load i of the k-block at byte offset ko, kOob past the end.  Where both marks meet, their sum
  // wraps to row kRows i of the region's first column, which is in range only if it is inside
  // the matrix; what it reads is used by nothing.
  static constexpr uint32_t load(uint32_t voff, uint32_t ko, int i, uint32_t ld2) {
    return voff + (ko + (uint32_t)(kRows * i) * ld2);
  }
};

}  // namespace moonep
