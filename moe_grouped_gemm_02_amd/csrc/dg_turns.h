// How the waves of a workgroup share a range of rows.  Host code too, and nothing of
// HIP: what it forms at the end of the 32-bit range can be checked by a host compiler.
#pragma once

namespace dg {

// Wave w of WAVES has rows from + w, from + w + WAVES, .. below `to`.  They are counted
// by what is left of the range: from + w and a row's successor may lie past 2^31 - 1
// and are formed only where they are rows.
template <int WAVES>
struct Turns {
  int to, left;  // left: rows from this one to the end, if any
  __host__ __device__ constexpr Turns(int from, int to_, int wave) : to(to_), left(to_ - from - wave) {}
  __host__ __device__ constexpr bool here() const { return left > 0; }
  __host__ __device__ constexpr int row() const { return to - left; }
  __host__ __device__ constexpr bool has_next() const { return left > WAVES; }
  __host__ __device__ constexpr int next_row() const { return to - (left - WAVES); }
  __host__ __device__ constexpr void next() { left -= WAVES; }
};

}  // namespace dg
