// linear_join.cuh -- how the CTAs of a cluster that share a tile of a product along K
// add up their partial sums.
#pragma once

#include "linear.cuh"
#include "umma.cuh"

namespace kda {

constexpr uint32_t kJoinRows = 128;  // channels of a tile

// This rank's columns of the tile, added up over R ranks in their order, and their epilogue
// finish(sums, column): a column per warp (of four) and four neighbouring channels per lane,
// several columns in flight.  The sums lie as [column][channel] at `part`, this lane's.
template <int R, typename F>
__device__ __forceinline__ void join(uint32_t part, uint32_t rank, int warp, int cols, const F& finish) {
  using namespace umma;
  constexpr int kFlight = R == 8 ? 2 : 4;
  uint32_t from[R];
#pragma unroll
  for (uint32_t r = 0; r < R; ++r) from[r] = map_to_rank(part, r);
  for (int c0 = rank + warp * R; c0 < cols; c0 += 4 * R * kFlight) {
    float4 v[kFlight][R];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int c = c0 + 4 * R * i < cols ? c0 + 4 * R * i : c0;
#pragma unroll
      for (int r = 0; r < R; ++r) v[i][r] = ld_cluster_f32x4(from[r] + c * kJoinRows * 4);
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      float4 z = v[i][0];
#pragma unroll
      for (int r = 1; r < R; ++r) {
        z.x += v[i][r].x; z.y += v[i][r].y; z.z += v[i][r].z; z.w += v[i][r].w;
      }
      const int c = c0 + 4 * R * i;
      if (c < cols) finish(z, c);
    }
  }
}
template <typename F>
__device__ __forceinline__ void join(uint32_t ranks, uint32_t part, uint32_t rank, int warp, int cols,
                                     const F& finish) {
  switch (ranks) {
    case 1: join<1>(part, rank, warp, cols, finish); break;
    case 2: join<2>(part, rank, warp, cols, finish); break;
    case 4: join<4>(part, rank, warp, cols, finish); break;
    default: join<8>(part, rank, warp, cols, finish); break;
  }
}

}  // namespace kda
