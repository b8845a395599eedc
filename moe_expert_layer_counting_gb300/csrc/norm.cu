// norm.cu -- the norms before and after the expert layer with its gate and
// residual scale, and their gradients (include/moe_norm.h has the formulas).
//
// Both directions are bound by HBM: every row is read once, kept in registers
// over its reductions and written once.  A block owns a row; its threads own
// 16-byte vectors of 8 values.
#include <cuda_bf16.h>

#include "../../include/moe_norm.h"
#include "host_common.h"
#include "ptx.cuh"

namespace mxq {

namespace {

constexpr int kMaxH = 16384;
constexpr int kMaxWarps = 32;
constexpr int kBackwardThreads = 512;
constexpr int kMaxParts = 304;         // blocks whose column sums the backward keeps apart

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 unpack_bf16x8(const uint4 &q) {
  F8 f;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFFu);
    f.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return f;
}

__device__ __forceinline__ uint4 pack_bf16x8(const F8 &f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.v[2 * i], f.v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values of a row as they lie in memory (registers until they are used).
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> {
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t *p) { q = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ F8 get() const { return unpack_bf16x8(q); }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ F8 get() const { return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};

__device__ __forceinline__ void store8(uint16_t *p, const F8 &f) { *reinterpret_cast<uint4 *>(p) = pack_bf16x8(f); }
__device__ __forceinline__ void store8(float *p, const F8 &f) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}

// Eight values of a weight or gate, of either type (the same branch for the
// whole launch).
__device__ __forceinline__ F8 load8_any(const void *p, int dtype, int64_t i) {
  if (dtype == MOE_BF16) return unpack_bf16x8(__ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i)));
  const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
  const float4 a = __ldg(q), b = __ldg(q + 1);
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ float load1_any(const void *p, int dtype, int64_t i) {
  return dtype == MOE_BF16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store1_any(void *p, int dtype, int64_t i, float v) {
  if (dtype == MOE_BF16)
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// Sums of N values over the block, the same bits in every thread (each adds
// the warps' sums in the same order).  One barrier; a buffer `red`
// [N][kMaxWarps] may be used again after another sum in another buffer.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *red) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warps = (int)(blockDim.x >> 5);
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * kMaxWarps + (threadIdx.x >> 5)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += red[i * kMaxWarps + w];
    v[i] = s;
  }
}

template <typename XT, int V>
__global__ void norm_forward_kernel(const moe_norm_args a) {
  __shared__ float red[2][kMaxWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int H = (int)a.H, vecs = H >> 3;
  const float inv_h = 1.0f / (float)H;
  const XT *x = static_cast<const XT *>(a.x) + t * a.ldx;
  const uint16_t *b = a.b ? a.b + t * a.ldb : nullptr;
  Raw8<XT> xr[V];
  Raw8<uint16_t> br[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (int)threadIdx.x + i * (int)blockDim.x;
    if (c < vecs) {
      xr[i].load(x + 8 * c);
      if (b) br[i].load(b + 8 * c);
    }
  }
  float gate_t = 1.0f;
  if (a.gate_kind == MOE_GATE_TOKEN) {
    gate_t = load1_any(a.gate, a.gate_dtype, t);
    if (a.gate_sigmoid) gate_t = sigmoid(gate_t);
  }
  float rb = 1.0f;
  if (b && a.w_post) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if ((int)threadIdx.x + i * (int)blockDim.x < vecs) {
        const F8 f = br[i].get();
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(f.v[j], f.v[j], s[0]);
      }
    }
    block_sum(s, red[0]);
    rb = __frsqrt_rn(s[0] * inv_h + a.eps);
  }
  F8 y[V];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (int)threadIdx.x + i * (int)blockDim.x;
    if (c < vecs) {
      y[i] = xr[i].get();
      if (b) {
        F8 u = br[i].get();
        if (a.w_post) {
          const F8 w = load8_any(a.w_post, a.w_dtype, 8 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) u.v[j] = u.v[j] * rb * (a.weight_offset + w.v[j]);
        }
        if (a.gate_kind >= MOE_GATE_CHANNEL) {
          const F8 g = load8_any(a.gate, a.gate_dtype, (a.gate_kind == MOE_GATE_FULL ? t * a.ld_gate : 0) + 8 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) u.v[j] *= a.gate_sigmoid ? sigmoid(g.v[j]) : g.v[j];
        } else if (a.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
          for (int j = 0; j < 8; ++j) u.v[j] *= gate_t;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i].v[j] = fmaf(a.residual_scale, y[i].v[j], u.v[j]);
        if (a.y) store8(static_cast<XT *>(a.y) + t * a.ldy + 8 * c, y[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(y[i].v[j], y[i].v[j], s[0]);
    }
  }
  if (!a.n) return;
  block_sum(s, red[1]);
  const float r = __frsqrt_rn(s[0] * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (int)threadIdx.x + i * (int)blockDim.x;
    if (c < vecs) {
      const F8 w = load8_any(a.w_pre, a.w_dtype, 8 * c);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i].v[j] = y[i].v[j] * r * (a.weight_offset + w.v[j]);
      store8(a.n + t * a.ldn + 8 * c, y[i]);
    }
  }
}

// Column sums over rows (dw_pre, dw_post, dgate of a channel gate): each block
// adds up its rows' values in registers, in row order, and leaves one part;
// norm_parts_kernel adds the parts in block order.
enum : int { kSumPre = 0, kSumPost = 1, kSumGate = 2 };

template <typename XT, int V>
__global__ void __launch_bounds__(kBackwardThreads) norm_backward_kernel(const moe_norm_args a, const moe_norm_grads g,
                                                                         float *parts) {
  __shared__ float red_buf[2][4 * kMaxWarps];      // of even and odd rows
  int turn = 0;
  pdl_launch_dependents();
  pdl_wait();
  const int H = (int)a.H, vecs = H >> 3;
  const float inv_h = 1.0f / (float)H;
  F8 sums[3][V];
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[k][i].v[j] = 0.f;

  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    float *red = red_buf[turn];
    const XT *y = static_cast<const XT *>(a.x) + t * a.ldx;
    Raw8<XT> yr[V], dyr[V];
    Raw8<uint16_t> br[V], dnr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (int)threadIdx.x + i * (int)blockDim.x;
      if (c < vecs) {
        if (a.w_pre) {
          yr[i].load(y + 8 * c);
          dnr[i].load(g.dn + t * g.ld_dn + 8 * c);
        }
        if (g.dy) dyr[i].load(static_cast<const XT *>(g.dy) + t * g.ld_dy + 8 * c);
        if (a.b) br[i].load(a.b + t * a.ldb + 8 * c);
      }
    }
    float gate_t = 1.0f;
    if (a.gate_kind == MOE_GATE_TOKEN) {
      gate_t = load1_any(a.gate, a.gate_dtype, t);
      if (a.gate_sigmoid) gate_t = sigmoid(gate_t);
    }
    // sums of y^2, dn w y and b^2
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (int)threadIdx.x + i * (int)blockDim.x;
      if (c < vecs) {
        if (a.w_pre) {
          const F8 f = yr[i].get(), d = dnr[i].get(), w = load8_any(a.w_pre, a.w_dtype, 8 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s[0] = fmaf(f.v[j], f.v[j], s[0]);
            s[1] = fmaf(d.v[j] * (a.weight_offset + w.v[j]), f.v[j], s[1]);
          }
        }
        if (a.b && a.w_post) {
          const F8 f = br[i].get();
#pragma unroll
          for (int j = 0; j < 8; ++j) s[2] = fmaf(f.v[j], f.v[j], s[2]);
        }
      }
    }
    block_sum(s, red);
    const float r = __frsqrt_rn(s[0] * inv_h + a.eps);
    const float rb = a.w_post ? __frsqrt_rn(s[2] * inv_h + a.eps) : 1.0f;
    const float back = r * r * s[1] * inv_h;              // mean(dn w h) r
    // d, and the sum of d g w_post b (token gates: without g)
    F8 d[V];
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (int)threadIdx.x + i * (int)blockDim.x;
      if (c < vecs) {
        if (g.dy) {
          d[i] = dyr[i].get();
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) d[i].v[j] = 0.f;
        }
        if (a.w_pre) {
          const F8 f = yr[i].get(), n = dnr[i].get(), w = load8_any(a.w_pre, a.w_dtype, 8 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            d[i].v[j] += r * (n.v[j] * (a.weight_offset + w.v[j]) - f.v[j] * back);
            sums[kSumPre][i].v[j] = fmaf(n.v[j], f.v[j] * r, sums[kSumPre][i].v[j]);
          }
        }
        if (g.dx) {
          F8 o = d[i];
          if (a.b)
#pragma unroll
            for (int j = 0; j < 8; ++j) o.v[j] *= a.residual_scale;
          store8(static_cast<XT *>(g.dx) + t * g.ld_dx + 8 * c, o);
        }
        if (a.b) {
          const F8 f = br[i].get();
          F8 w;
          if (a.w_post) {
            w = load8_any(a.w_post, a.w_dtype, 8 * c);
#pragma unroll
            for (int j = 0; j < 8; ++j) w.v[j] = (w.v[j] + a.weight_offset) * rb;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w.v[j] = 1.0f;
          }
          if (a.gate_kind >= MOE_GATE_CHANNEL) {
            const bool full = a.gate_kind == MOE_GATE_FULL;
            F8 z = load8_any(a.gate, a.gate_dtype, (full ? t * a.ld_gate : 0) + 8 * c);
            F8 dz;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float gv = a.gate_sigmoid ? sigmoid(z.v[j]) : z.v[j];
              dz.v[j] = d[i].v[j] * f.v[j] * w.v[j];
              if (full && a.gate_sigmoid) dz.v[j] *= gv * (1.0f - gv);
              d[i].v[j] *= gv;
            }
            if (full) {
              if (g.dgate) {
                if (a.gate_dtype == MOE_BF16)
                  store8(static_cast<uint16_t *>(g.dgate) + t * g.ld_dgate + 8 * c, dz);
                else
                  store8(static_cast<float *>(g.dgate) + t * g.ld_dgate + 8 * c, dz);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) sums[kSumGate][i].v[j] += dz.v[j];
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) q[0] = fmaf(d[i].v[j] * w.v[j], f.v[j], q[0]);
        }
      }
    }
    if (!a.b) continue;
    if (a.w_post || a.gate_kind == MOE_GATE_TOKEN) block_sum(q, red + 3 * kMaxWarps);
    if (a.gate_kind == MOE_GATE_TOKEN && g.dgate && threadIdx.x == 0)
      store1_any(g.dgate, a.gate_dtype, t, a.gate_sigmoid ? q[0] * gate_t * (1.0f - gate_t) : q[0]);
    // db = rb (g d w - h mean(g d w h)); w above carries rb once, so with
    // q = sum(g d w rb b):  db = g d w rb - b rb^2 q / H
    const float back_b = a.w_post ? rb * rb * q[0] * inv_h * (a.gate_kind == MOE_GATE_TOKEN ? gate_t : 1.0f) : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (int)threadIdx.x + i * (int)blockDim.x;
      if (c < vecs) {
        const F8 f = br[i].get();
        F8 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = d[i].v[j] * gate_t;
        if (a.w_post) {
          const F8 w = load8_any(a.w_post, a.w_dtype, 8 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sums[kSumPost][i].v[j] = fmaf(o.v[j], f.v[j] * rb, sums[kSumPost][i].v[j]);
            o.v[j] = o.v[j] * (w.v[j] + a.weight_offset) * rb - f.v[j] * back_b;
          }
        }
        if (g.db) store8(g.db + t * g.ld_db + 8 * c, o);
      }
    }
  }
  float *part = parts + (int64_t)blockIdx.x * 3 * H;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (int)threadIdx.x + i * (int)blockDim.x;
    if (c < vecs) {
      if (g.dw_pre) store8(part + kSumPre * H + 8 * c, sums[kSumPre][i]);
      if (g.dw_post) store8(part + kSumPost * H + 8 * c, sums[kSumPost][i]);
      if (a.gate_kind == MOE_GATE_CHANNEL && g.dgate) store8(part + kSumGate * H + 8 * c, sums[kSumGate][i]);
    }
  }
}

// blockIdx.y: which sum; 32 columns per block, eight threads per column.
__global__ void __launch_bounds__(256) norm_parts_kernel(const moe_norm_args a, const moe_norm_grads g,
                                                         const float *parts, int n) {
  __shared__ float red[8][33];
  pdl_launch_dependents();
  pdl_wait();
  const int H = (int)a.H, which = blockIdx.y;
  const bool wanted = which == kSumPre ? g.dw_pre != nullptr
                      : which == kSumPost ? g.dw_post != nullptr
                                          : a.gate_kind == MOE_GATE_CHANNEL && g.dgate != nullptr;
  if (!wanted) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float s = 0.f;
  if (c < H)
    for (int p = k; p < n; p += 8) s += parts[((int64_t)p * 3 + which) * H + c];
  red[k][threadIdx.x & 31] = s;
  __syncthreads();
  if (k != 0 || c >= H) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
  if (which == kSumPre) {
    g.dw_pre[c] = s;
  } else if (which == kSumPost) {
    g.dw_post[c] = s;
  } else {
    if (a.gate_sigmoid) {
      const float v = sigmoid(load1_any(a.gate, a.gate_dtype, c));
      s *= v * (1.0f - v);
    }
    store1_any(g.dgate, a.gate_dtype, c, s);
  }
}

// ---------------------------------------------------------------- host

bool dtype_ok(int32_t d) { return d == MOE_BF16 || d == MOE_F32; }

// A row tensor that has to be there.
int check_row(const void *p, int64_t ld, int64_t H) {
  if (!p || ld < H) return MOE_ERR_INVALID_ARG;
  if (ld % 8 != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  return aligned(p, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}

int check_norm(const moe_norm_args *a) {
  if (!a || a->struct_size != sizeof(moe_norm_args)) return MOE_ERR_INVALID_ARG;
  if (a->T < 0 || a->H <= 0 || !dtype_ok(a->x_dtype) || !dtype_ok(a->w_dtype) || !(a->eps >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (a->gate_kind < MOE_GATE_NONE || a->gate_kind > MOE_GATE_FULL || (a->gate_sigmoid != 0 && a->gate_sigmoid != 1))
    return MOE_ERR_INVALID_ARG;
  if (a->H % 8 != 0 || a->H > kMaxH || a->T > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (a->T == 0) return MOE_OK;        // row tensors may be null
  if ((a->gate_kind != MOE_GATE_NONE) != (a->gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!a->b && (a->gate || a->w_post || !a->w_pre)) return MOE_ERR_INVALID_ARG;
  if (a->gate && !dtype_ok(a->gate_dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->w_post, 16) || !aligned(a->w_pre, 16)) return MOE_ERR_MISALIGNED;
  if (a->gate && !aligned(a->gate, a->gate_kind == MOE_GATE_TOKEN ? (a->gate_dtype == MOE_F32 ? 4 : 2) : 16))
    return MOE_ERR_MISALIGNED;
  int rc = check_row(a->x, a->ldx, a->H);
  if (rc == MOE_OK && a->b) rc = check_row(a->b, a->ldb, a->H);
  if (rc == MOE_OK && a->gate_kind == MOE_GATE_FULL) rc = check_row(a->gate, a->ld_gate, a->H);
  return rc;
}

struct Shape {
  int threads, v;      // threads per row, vectors per thread (1, 2 or 4)
};

// Threads of a row: `v` vectors each, in whole warps.
Shape row_shape(int64_t H, int v, int most) {
  const int vecs = (int)(H / 8);
  while (v < 4 && (vecs + v - 1) / v > most) v *= 2;
  return {(int)round_up((size_t)((vecs + v - 1) / v), 32), v};
}

template <typename XT>
int forward_launch(const moe_norm_args &a, cudaStream_t st) {
  const Shape s = row_shape(a.H, a.T <= 4 * num_sms() ? 1 : 4, 1024);
  auto kernel = s.v == 1 ? norm_forward_kernel<XT, 1> : s.v == 2 ? norm_forward_kernel<XT, 2> : norm_forward_kernel<XT, 4>;
  return launch_pdl(kernel, dim3((unsigned)a.T), dim3(s.threads), 0, st, a);
}

int backward_parts(int64_t T) { return (int)std::min<int64_t>(T, std::min(2 * num_sms(), kMaxParts)); }

template <typename XT>
int backward_launch(const moe_norm_args &a, const moe_norm_grads &g, cudaStream_t st) {
  const Shape s = row_shape(a.H, 2, kBackwardThreads);
  float *parts = static_cast<float *>(g.workspace);
  auto kernel = s.v == 2 ? norm_backward_kernel<XT, 2> : norm_backward_kernel<XT, 4>;
  const int n = backward_parts(a.T);
  const int rc = launch_pdl(kernel, dim3(n), dim3(s.threads), 0, st, a, g, parts);
  if (rc != MOE_OK) return rc;
  const bool gate = a.gate_kind == MOE_GATE_CHANNEL && g.dgate;
  if (!g.dw_pre && !g.dw_post && !gate) return MOE_OK;
  return launch_pdl(norm_parts_kernel, dim3((unsigned)ceil_div(a.H, 32), gate ? 3 : g.dw_post ? 2 : 1), dim3(256), 0, st,
                    a, g, static_cast<const float *>(parts), n);
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" int moe_norm_forward(const moe_norm_args *a, cudaStream_t stream) {
  int rc = check_norm(a);
  if (rc != MOE_OK || a->T == 0) return rc;
  if ((a->w_pre != nullptr) != (a->n != nullptr) || (!a->b && a->y) || (a->b && !a->y && !a->n)) return MOE_ERR_INVALID_ARG;
  if (a->y && (rc = check_row(a->y, a->ldy, a->H)) != MOE_OK) return rc;
  if (a->n && (rc = check_row(a->n, a->ldn, a->H)) != MOE_OK) return rc;
  return a->x_dtype == MOE_F32 ? forward_launch<float>(*a, stream) : forward_launch<uint16_t>(*a, stream);
}

extern "C" size_t moe_norm_workspace_size(int64_t T, int64_t H) {
  if (T < 0 || H <= 0 || H > kMaxH) return 0;
  return round_up((size_t)std::min<int64_t>(T, kMaxParts) * 3 * (size_t)H * 4, 256) + 256;
}

extern "C" int moe_norm_backward(const moe_norm_args *a, const moe_norm_grads *g, cudaStream_t stream) {
  int rc = check_norm(a);
  if (rc != MOE_OK) return rc;
  if (!g || g->struct_size != sizeof(moe_norm_grads)) return MOE_ERR_INVALID_ARG;
  if (!aligned(g->dw_pre, 16) || !aligned(g->dw_post, 16) || !aligned(g->dgate, 4)) return MOE_ERR_MISALIGNED;
  if (!g->workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned(g->workspace, 256)) return MOE_ERR_MISALIGNED;
  if (g->workspace_bytes < moe_norm_workspace_size(a->T, a->H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (a->T == 0) {
    const size_t w = (size_t)a->H * 4;
    if (g->dw_pre && cudaMemsetAsync(g->dw_pre, 0, w, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (g->dw_post && cudaMemsetAsync(g->dw_post, 0, w, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (g->dgate && a->gate_kind == MOE_GATE_CHANNEL &&
        cudaMemsetAsync(g->dgate, 0, a->gate_dtype == MOE_F32 ? w : w / 2, stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if ((a->w_pre != nullptr) != (g->dn != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((g->dw_pre && !a->w_pre) || (g->dw_post && !a->w_post) || (g->db && !a->b) || (g->dgate && !a->gate))
    return MOE_ERR_INVALID_ARG;
  if (g->dy && (rc = check_row(g->dy, g->ld_dy, a->H)) != MOE_OK) return rc;
  if (g->dn && (rc = check_row(g->dn, g->ld_dn, a->H)) != MOE_OK) return rc;
  if (g->dx && (rc = check_row(g->dx, g->ld_dx, a->H)) != MOE_OK) return rc;
  if (g->db && (rc = check_row(g->db, g->ld_db, a->H)) != MOE_OK) return rc;
  if (g->dgate && a->gate_kind == MOE_GATE_FULL && (rc = check_row(g->dgate, g->ld_dgate, a->H)) != MOE_OK) return rc;
  return a->x_dtype == MOE_F32 ? backward_launch<float>(*a, *g, stream) : backward_launch<uint16_t>(*a, *g, stream);
}
