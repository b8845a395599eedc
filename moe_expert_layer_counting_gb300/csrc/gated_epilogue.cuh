// gated_epilogue.cuh -- epilogues of the grouped products that carry the gated
// activation (include/moe_gated.h), and the exchange between lanes that turns
// accumulators into rows.
//
// An activation is f(z) = z s(q(z)) with s(q) = 1 / (1 + exp(-q)):
//   SiLU       q = z
//   GELU(tanh) q = 2 sqrt(2/pi) (z + 0.044715 z^3), as 1 + tanh(u) = 2 s(2u)
// and f'(z) = s + z s (1 - s) q'(z).
//
// exp and the quotient are the fast ones (a few units of 2^-23, against 2^-8
// of the BF16 outputs and 1e-6 of a sum over a row); quotients beyond 2^126 flush to 0.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "../../include/moe_gated.h"
#include "ptx.cuh"

namespace mxq {

namespace {

struct GatedArgs {
  int I, activation;
  const float *row_w;     // or NULL
  uint16_t *a;            // gated: out or NULL; gradient: in
  int64_t ld_a;
  uint16_t *h;            // gradient: or NULL
  int64_t ld_h;
  uint16_t *da;
  int64_t ld_da;
  float *part;            // gradient: sums of dh f up over 32 columns, [I / 32][P], or NULL
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// N values (float bits) of rows 0 .. N-1 in each lane, a lane a column.  Three
// exchanges between lanes (of one value, one word, two words) turn them so that
// lane l holds columns 8 (l / 8) .. + 7 of rows 8 r + l % 8 as 16 bytes of BF16,
// handed to put(r, piece).
template <int N, typename V, typename Put>
__device__ __forceinline__ void turn_bf16(const V (&v)[N], int lane, Put put) {
  const bool b0 = (lane & 1) != 0, b1 = (lane & 2) != 0, b2 = (lane & 4) != 0;
  auto as_float = [](V x) {
    if constexpr (sizeof(V) == 4 && !std::is_same<V, float>::value)
      return __uint_as_float(x);
    else
      return x;
  };
  uint32_t w[N / 2];                   // rows 2 p + b0, two columns
#pragma unroll
  for (int p = 0; p < N / 2; ++p) {
    const float a = as_float(v[2 * p]), b = as_float(v[2 * p + 1]);
    const float got = __shfl_xor_sync(0xffffffffu, b0 ? a : b, 1);
    w[p] = b0 ? pack_bf16(got, b) : pack_bf16(a, got);
  }
  uint32_t u[N / 4][2];                // rows 4 q + 2 b1 + b0, four columns
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? w[2 * q] : w[2 * q + 1], 2);
    u[q][0] = b1 ? got : w[2 * q];
    u[q][1] = b1 ? w[2 * q + 1] : got;
  }
#pragma unroll
  for (int r = 0; r < N / 8; ++r) {
    const uint32_t got0 = __shfl_xor_sync(0xffffffffu, b2 ? u[2 * r][0] : u[2 * r + 1][0], 4);
    const uint32_t got1 = __shfl_xor_sync(0xffffffffu, b2 ? u[2 * r][1] : u[2 * r + 1][1], 4);
    put(r, b2 ? make_uint4(got0, got1, u[2 * r + 1][0], u[2 * r + 1][1])
              : make_uint4(u[2 * r][0], u[2 * r][1], got0, got1));
  }
}

// As turn_bf16 for eight rows, with the values left in float32: t[c] is column 8 (l / 8) + c of row l % 8.
__device__ __forceinline__ void turn_f32(const uint32_t (&v)[8], int lane, float (&t)[8]) {
  const bool b0 = (lane & 1) != 0, b1 = (lane & 2) != 0, b2 = (lane & 4) != 0;
  float w[4][2];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float a = __uint_as_float(v[2 * p]), b = __uint_as_float(v[2 * p + 1]);
    const float got = __shfl_xor_sync(0xffffffffu, b0 ? a : b, 1);
    w[p][0] = b0 ? got : a;
    w[p][1] = b0 ? b : got;
  }
  float u[2][4];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float got = __shfl_xor_sync(0xffffffffu, b1 ? w[2 * q][i] : w[2 * q + 1][i], 2);
      u[q][i] = b1 ? got : w[2 * q][i];
      u[q][2 + i] = b1 ? w[2 * q + 1][i] : got;
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float got = __shfl_xor_sync(0xffffffffu, b2 ? u[0][i] : u[1][i], 4);
    t[i] = b2 ? got : u[0][i];
    t[4 + i] = b2 ? u[1][i] : got;
  }
}

// s(q(z)) and q'(z).  GELU's q is taken at |z| <= 12, past which s is 0 or 1 in
// float32, so that no power of z overflows.
__device__ __forceinline__ float gate_sigmoid(int activation, float z, float &dq) {
  float q = z;
  dq = 1.f;
  if (activation == MOE_ACT_GELU_TANH) {
    constexpr float kRoot = 1.5957691216057308f;       // 2 sqrt(2 / pi)
    const float c = fminf(fmaxf(z, -12.f), 12.f), cc = c * c;
    q = kRoot * c * fmaf(0.044715f, cc, 1.f);
    dq = kRoot * fmaf(3.f * 0.044715f, cc, 1.f);
  }
  return __fdividef(1.f, 1.f + __expf(-q));
}

// Gated forward: 32 N slots of this warp's 32 lanes, which hold columns
// col0 .. + 15 as 8 gate rows, 8 up rows, 8 gate rows, 8 up rows of the weights.
// Gate and up of a column lie 8 lanes apart; the gate's lane takes the first 16
// rows of both, the up's lane the others.
__device__ __forceinline__ void gated_rows(const uint32_t (&v)[32], int64_t row0, int rows, int col0, const GatedArgs &g,
                                           int lane) {
  const bool is_up = (lane & 8) != 0;
  const int col = col0 + 8 * (lane >> 4);
  if (g.a)
    turn_bf16<32>(v, lane, [&](int r, const uint4 &piece) {
      const int row = 8 * r + (lane & 7);
      if (row < rows && col < g.I)
        *reinterpret_cast<uint4 *>(g.a + (row0 + row) * g.ld_a + (is_up ? g.I : 0) + col) = piece;
    });
  const float w = g.row_w && lane < rows ? __ldg(g.row_w + row0 + lane) : 1.f;
  float h[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    const float low = __uint_as_float(v[t]), high = __uint_as_float(v[16 + t]);
    const float got = __shfl_xor_sync(0xffffffffu, is_up ? low : high, 8);
    const float wt = __shfl_sync(0xffffffffu, w, t + (is_up ? 16 : 0));
    const float gate = is_up ? got : low, up = is_up ? high : got;
    float dq;
    h[t] = gate * gate_sigmoid(g.activation, gate, dq) * up * wt;
  }
  turn_bf16<16>(h, lane, [&](int r, const uint4 &piece) {
    const int row = 8 * r + (lane & 7) + (is_up ? 16 : 0);
    if (row < rows && col < g.I) *reinterpret_cast<uint4 *>(g.h + (row0 + row) * g.ld_h + col) = piece;
  });
}

// The way back, for eight N slots (`rows` of them rows, from row0) at this warp's 32 columns from col0: what a lane reads of a,
// and these slots of dh.
struct GatedRow {
  uint4 gate, up;

  __device__ __forceinline__ void take(int64_t row0, int rows, int col0, const GatedArgs &g, int lane) {
    const int col = col0 + 8 * (lane >> 3), row = lane & 7;
    gate = up = make_uint4(0, 0, 0, 0);
    if (row < rows && col < g.I) {
      const uint16_t *a = g.a + (row0 + row) * g.ld_a + col;
      gate = *reinterpret_cast<const uint4 *>(a);
      up = *reinterpret_cast<const uint4 *>(a + g.I);
    }
  }
};

__device__ __forceinline__ void gated_grad_rows(const uint32_t (&v)[8], const GatedRow &in, int64_t row0, int rows, int col0, int64_t P,
                                                const GatedArgs &g, int lane) {
  const int col = col0 + 8 * (lane >> 3), row = lane & 7;
  const bool mine = row < rows && col < g.I;
  float t[8];
  turn_f32(v, lane, t);
  const float w = g.row_w && mine ? __ldg(g.row_w + row0 + row) : 1.f;
  const uint32_t gw[4] = {in.gate.x, in.gate.y, in.gate.z, in.gate.w};
  const uint32_t uw[4] = {in.up.x, in.up.y, in.up.z, in.up.w};
  uint32_t dg[4], du[4], hh[4];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a[2], b[2], c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float z = __uint_as_float(k == 0 ? gw[i] << 16 : gw[i] & 0xFFFF0000u);
      const float u = __uint_as_float(k == 0 ? uw[i] << 16 : uw[i] & 0xFFFF0000u);
      float dq;
      const float s = gate_sigmoid(g.activation, z, dq);
      const float f = z * s;
      const float d = t[2 * i + k];
      sum = fmaf(d * f, u, sum);
      const float dw = d * w;
      a[k] = dw * u * fmaf(f * (1.f - s), dq, s);
      b[k] = dw * f;
      c[k] = f * u * w;
    }
    dg[i] = pack_bf16(a[0], a[1]);
    du[i] = pack_bf16(b[0], b[1]);
    hh[i] = pack_bf16(c[0], c[1]);
  }
  if (mine) {
    uint16_t *da = g.da + (row0 + row) * g.ld_da + col;
    *reinterpret_cast<uint4 *>(da) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
    *reinterpret_cast<uint4 *>(da + g.I) = make_uint4(du[0], du[1], du[2], du[3]);
    if (g.h) *reinterpret_cast<uint4 *>(g.h + (row0 + row) * g.ld_h + col) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
  }
  if (g.part) {
    if (!mine) sum = 0.f;              // a row of another expert, or columns past the last
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (lane < 8 && row < rows) g.part[(int64_t)(col0 >> 5) * P + row0 + row] = sum;
  }
}

}  // namespace

}  // namespace mxq
