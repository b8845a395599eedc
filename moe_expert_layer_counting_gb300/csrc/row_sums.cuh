// row_sums.cuh -- sums over the warps that own a row, of the norms' kernels.
#pragma once
#include <cstdint>

namespace mxq {

// Sums of up to four values over `warps` warps (at most 32), the same bits in
// every thread.  Lanes hand values on as they add (6 shuffles for four values
// instead of 20), every warp adds the warps' sums in the same tree; the result
// of value k is in `v[k]`.  `sync` joins the warps, once; `red` [4][32] may be
// used again after another sum in another buffer.
template <int N, typename Sync>
__device__ __forceinline__ void group_sum(float (&v)[N], int warps, int warp, float *red, Sync sync) {
  static_assert(N >= 1 && N <= 4, "one to four values");
  const int lane = (int)(threadIdx.x & 31);
  float s;
  if (N == 1) {
    s = v[0];
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    s += __shfl_xor_sync(0xffffffffu, s, 8);
  } else {
    // lanes with bit 4 keep values 2 and 3, then lanes with bit 3 the odd one
    const float v1 = v[1 % N], v2 = N > 2 ? v[2 % N] : 0.f, v3 = N > 3 ? v[3 % N] : 0.f;
    const bool up = (lane & 16) != 0;
    float a = (up ? v2 : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v2, 16);
    float b = (up ? v3 : v1) + __shfl_xor_sync(0xffffffffu, up ? v1 : v3, 16);
    const bool odd = (lane & 8) != 0;
    s = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
  }
  s += __shfl_xor_sync(0xffffffffu, s, 4);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  if (warps > 1) {
    // [value][warp]; absent warps were zeroed once
    if ((lane & 7) == 0 && (N > 1 || lane == 0)) red[(lane >> 3) * 32 + warp] = s;
    sync();
    const float4 q = *reinterpret_cast<const float4 *>(red + (N == 1 ? 0 : (lane >> 3) * 32) + 4 * (lane & 7));
    s = (q.x + q.y) + (q.z + q.w);
    s += __shfl_xor_sync(0xffffffffu, s, 4);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
  } else {
    sync();
  }
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, s, N == 1 ? 0 : 8 * k);
}

// As group_sum, of three values of each of R rows; `red` [R][4][32], one sync.
template <int R, typename Sync>
__device__ __forceinline__ void group_sums(float (&v)[R][3], int warps, int warp, float *red, Sync sync) {
  const int lane = (int)(threadIdx.x & 31);
  const bool up = (lane & 16) != 0, odd = (lane & 8) != 0;
  float s[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float a = (up ? v[j][2] : v[j][0]) + __shfl_xor_sync(0xffffffffu, up ? v[j][0] : v[j][2], 16);
    float b = (up ? 0.f : v[j][1]) + __shfl_xor_sync(0xffffffffu, up ? v[j][1] : 0.f, 16);
    s[j] = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1)
#pragma unroll
    for (int j = 0; j < R; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
  if (warps > 1) {
    if ((lane & 7) == 0)
#pragma unroll
      for (int j = 0; j < R; ++j) red[j * 128 + (lane >> 3) * 32 + warp] = s[j];
    sync();
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float4 q = *reinterpret_cast<const float4 *>(red + j * 128 + (lane >> 3) * 32 + 4 * (lane & 7));
      s[j] = (q.x + q.y) + (q.z + q.w);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < R; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
  } else {
    sync();
  }
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int k = 0; k < 3; ++k) v[j][k] = __shfl_sync(0xffffffffu, s[j], 8 * k);
}

}  // namespace mxq
