// Rotary positions with several axes, alone and with the RMS norm of every
// head's queries and keys in the same pass, forward and backward.
//
//   rotation   pair j of a token at positions p turns by a = p[axis_j] f_j:
//              (u, v) -> (u cos a - v sin a, u sin a + v cos a); the gradient
//              is the rotation by -a
//   norm       n_d = x_d r w_d, r = 1 / sqrt(mean_d x_d^2 + eps), y = R n
//   backward   g = R^T dy; dx_d = r (g_d w_d - x_d r^2 mean_e(g_e w_e x_e));
//              dw_d = sum over rows of g_d x_d r
//
// r is recomputed from x, which the backward reads anyway, so nothing is
// saved. Everything between the loads and the stores is fp32 and rounded
// once; the angles are formed in fp64 as turns (p f / 2 pi), reduced to
// [-1/2, 1/2] there, and only then handed to the fp32 sine and cosine:
// a position of 10^6 would otherwise cost the angle 20 of its 24 bits.
//
// Bound by HBM: a row is read once and written once (the norm's backward
// reads x and dy). A lane moves 8 channels, a power of two of lanes a row, and
// a thread keeps one (token, 8 channels) place for all heads of its unit, so
// an angle is computed once for 24 or 80 rows of it. A unit is a tile of
// tokens by a group of heads; the grid holds the blocks that fit on the GPU
// and each strides over the units, the number of head groups being the one
// whose longest block is shortest (plan_units).
//
// The weight gradients are summed per thread over its rows, per block through
// shared memory, and over the blocks by a second kernel, always in the same
// order: no atomics, the same bits every time.
#include <cuda_fp16.h>

#include "vsa_common.cuh"

namespace vsa {

namespace {

constexpr int kThreads = 256;

template <typename T>
struct Row8;  // 8 channels as they lie in memory
template <>
struct Row8<float> {
  static constexpr int REGS = 8;
  uint32_t r[8];
};
template <>
struct Row8<__nv_bfloat16> {
  static constexpr int REGS = 4;
  uint32_t r[4];
};
template <>
struct Row8<__half> {
  static constexpr int REGS = 4;
  uint32_t r[4];
};

template <typename T>
__device__ __forceinline__ Row8<T> load8(const T* p) {
  Row8<T> v;
#pragma unroll
  for (int i = 0; i < Row8<T>::REGS; i += 4) {
    const uint4 x = *(reinterpret_cast<const uint4*>(p) + i / 4);
    v.r[i] = x.x, v.r[i + 1] = x.y, v.r[i + 2] = x.z, v.r[i + 3] = x.w;
  }
  return v;
}

__device__ __forceinline__ void unpack(const Row8<float>& v, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v.r[i]);
}
__device__ __forceinline__ void unpack(const Row8<__nv_bfloat16>& v, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v.r[i] << 16);
    x[2 * i + 1] = __uint_as_float(v.r[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Row8<__half>& v, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v.r[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()), pack2(x[4], x[5], T()), pack2(x[6], x[7], T()));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Sum over the L lanes of a row.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One thread's place in a tile and its rotation coefficients.
template <typename T, int L, bool INTER>
struct Place {
  int lane_row, chunk;      // row of the tile, 8-channel chunk of the row
  bool in_row;              // the chunk lies inside D
  int partner;              // lane that holds the other half of the pairs (half-split)
  float sign;               // half-split: sign of the partner's sine term (first half: -1)
  uint32_t turned;          // bit i: channel i of the chunk is rotated
  float c[8], s[8];         // cosine, and the sine with the sign of y_i = x_i c_i + x'_i s_i

  __device__ __forceinline__ void init(int D, int rot) {
    lane_row = threadIdx.x / L;
    chunk = threadIdx.x % L;
    in_row = chunk * 8 < D;
    const int left = rot - chunk * 8;
    turned = left >= 8 ? 0xffu : left > 0 ? (1u << left) - 1u : 0u;
    partner = threadIdx.x & 31;
    sign = 1.f;
    if (!INTER && turned) {  // rot is a multiple of 16 here: a chunk lies in one half
      const int half = rot / 16;
      partner += chunk < half ? half : -half;
      sign = chunk < half ? -1.f : 1.f;
    }
  }

  // Coefficients for the token's positions (as fp64, one per axis). `back`
  // turns the other way.
  __device__ __forceinline__ void angles(const double* freq, const int* axis, const double (&pos)[kRopeAxes], int rot,
                                         bool back) {
    const float dir = back ? -1.f : 1.f;
    if (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = 1.f;
        s[2 * i] = s[2 * i + 1] = 0.f;
        if (turned >> (2 * i) & 1u) {
          float sn, cs;
          turn(freq, axis, pos, chunk * 4 + i, &sn, &cs);
          c[2 * i] = c[2 * i + 1] = cs;
          s[2 * i] = -dir * sn;
          s[2 * i + 1] = dir * sn;
        }
      }
    } else {
      const int first = (chunk * 8) % (rot > 0 ? rot / 2 : 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
        if (turned) {
          float sn, cs;
          turn(freq, axis, pos, first + i, &sn, &cs);
          c[i] = cs;
          s[i] = sign * dir * sn;
        }
      }
    }
  }

  __device__ __forceinline__ static void turn(const double* freq, const int* axis, const double (&pos)[kRopeAxes],
                                              int j, float* sn, float* cs) {
    const int a = axis[j];
    const double p = a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
    const double turns = p * freq[j];
    sincospif(2.f * (float)(turns - rint(turns)), sn, cs);
  }

  // The other channel of each pair (0 where a channel is not rotated, so that
  // an infinity there meets no zero coefficient).
  __device__ __forceinline__ void other(const Row8<T>& raw, const float (&x)[8], float (&xp)[8]) const {
    if (INTER) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xp[i] = turned >> i & 1u ? x[i ^ 1] : 0.f;
    } else {
      Row8<T> o;
#pragma unroll
      for (int i = 0; i < Row8<T>::REGS; ++i) o.r[i] = __shfl_sync(0xffffffffu, raw.r[i], partner);
      unpack(o, xp);
      if (!turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) xp[i] = 0.f;
      }
    }
  }
};

// The token's positions: the raster grid's (t, h, w), or the caller's list.
__device__ __forceinline__ void token_positions(const RopeParams& p, int b, int n, double (&pos)[kRopeAxes]) {
#pragma unroll
  for (int a = 0; a < kRopeAxes; ++a) pos[a] = 0.0;
  if (p.pos_kind == 0) {
    const unsigned un = n, uw = p.W, uh = p.H;
    const unsigned th = un / uw, t = th / uh;
    pos[0] = (double)((long long)t + p.origin[0]);
    pos[1] = (double)((long long)(th - t * uh) + p.origin[1]);
    pos[2] = (double)((long long)(un - th * uw) + p.origin[2]);
  } else {
    const long long o = (long long)b * p.pos_batch + (long long)n * p.axes;
#pragma unroll
    for (int a = 0; a < kRopeAxes; ++a)
      if (a < p.axes)
        pos[a] = p.pos_kind == 1 ? (double)static_cast<const int*>(p.pos)[o + a]
                                 : (double)static_cast<const float*>(p.pos)[o + a];
  }
}

// Frequencies (in turns) and axes from the launch parameters to shared memory.
__device__ __forceinline__ void stage_rotation(const RopeParams& p, double* freq, int* axis) {
  for (int j = threadIdx.x; j < p.rot / 2; j += kThreads) {
    freq[j] = p.freq[j];
    axis[j] = p.axis[j];
  }
  __syncthreads();
}

// U heads' rows in flight at a time.
template <typename T, int L, bool INTER, int U>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ double freq[kRopePairs];
  __shared__ int axis[kRopePairs];
  stage_rotation(p, freq, axis);
  Place<T, L, INTER> me;
  me.init(p.D, p.rot);
  constexpr int ROWS = kThreads / L;
  const float inv_d = 1.f / (float)p.D;
  for (long long u = blockIdx.x; u < p.units; u += gridDim.x) {
    const int g = (int)(u % p.groups);
    const long long bt = u / p.groups;
    const int b = (int)(bt / p.tiles), n = (int)(bt % p.tiles) * ROWS + me.lane_row;
    const bool live = n < p.N && me.in_row;
    double pos[kRopeAxes];
    token_positions(p, b, n < p.N ? n : 0, pos);
    me.angles(freq, axis, pos, p.rot, p.back != 0);
    const int total = p.t[0].heads + p.t[1].heads;
    const int h_lo = (int)((long long)total * g / p.groups), h_hi = (int)((long long)total * (g + 1) / p.groups);
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const RopeTensor& x = p.t[t];
      const int first = t ? p.t[0].heads : 0;
      const int lo = max(h_lo - first, 0), hi = min(h_hi - first, x.heads);
      if (lo >= hi) continue;
      // y_i = r (x_i A_i + x'_i B_i), the weight folded into A and B
      float A[8], B[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) A[i] = me.c[i], B[i] = me.s[i];
      if (x.w && me.in_row) {
        const float4 w0 = reinterpret_cast<const float4*>(x.w + me.chunk * 8)[0];
        const float4 w1 = reinterpret_cast<const float4*>(x.w + me.chunk * 8)[1];
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          A[i] *= w[i];
          if (INTER) B[i] *= w[i ^ 1];
        }
        if (!INTER && me.turned) {
          const int pc = me.chunk + (me.partner - (int)(threadIdx.x & 31));
          const float4 v0 = reinterpret_cast<const float4*>(x.w + pc * 8)[0];
          const float4 v1 = reinterpret_cast<const float4*>(x.w + pc * 8)[1];
          const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) B[i] *= v[i];
        }
      }
      const T* src = static_cast<const T*>(x.in) + b * x.in_b + n * x.in_n + me.chunk * 8;
      T* dst = static_cast<T*>(x.out) + b * x.out_b + n * x.out_n + me.chunk * 8;
#pragma unroll 1
      for (int h0 = lo; h0 < hi; h0 += U) {
        Row8<T> raw[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          raw[k] = Row8<T>{};
          if (live && h0 + k < hi) raw[k] = load8(src + (h0 + k) * x.in_h);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          float v[8], o[8];
          unpack(raw[k], v);
          me.other(raw[k], v, o);
          float r = 1.f;
          if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
            r = rsqrtf(fmaf(row_sum<L>(ss), inv_d, p.eps));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = r * fmaf(o[i], B[i], v[i] * A[i]);
          if (live && h0 + k < hi) store8(dst + (h0 + k) * x.out_h, v);
        }
      }
    }
  }
}

// Backward of the norm with the rotation: x.in = x, x.dy = dy, x.out = dx, the
// block's weight gradients to p.partial[block][tensor][D].
template <typename T, int L, bool INTER, int U>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_backward_kernel(const __grid_constant__ RopeParams p) {
  __shared__ double freq[kRopePairs];
  __shared__ int axis[kRopePairs];
  __shared__ float part[kThreads * 8];
  stage_rotation(p, freq, axis);
  Place<T, L, INTER> me;
  me.init(p.D, p.rot);
  constexpr int ROWS = kThreads / L;
  const float inv_d = 1.f / (float)p.D;
  float acc[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
  for (long long u = blockIdx.x; u < p.units; u += gridDim.x) {
    const int g = (int)(u % p.groups);
    const long long bt = u / p.groups;
    const int b = (int)(bt / p.tiles), n = (int)(bt % p.tiles) * ROWS + me.lane_row;
    const bool live = n < p.N && me.in_row;
    double pos[kRopeAxes];
    token_positions(p, b, n < p.N ? n : 0, pos);
    me.angles(freq, axis, pos, p.rot, true);
    const int total = p.t[0].heads + p.t[1].heads;
    const int h_lo = (int)((long long)total * g / p.groups), h_hi = (int)((long long)total * (g + 1) / p.groups);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const RopeTensor& x = p.t[t];
      const int first = t ? p.t[0].heads : 0;
      const int lo = max(h_lo - first, 0), hi = min(h_hi - first, x.heads);
      if (lo >= hi) continue;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = x.w && me.in_row ? x.w[me.chunk * 8 + i] : 1.f;
      const T* src = static_cast<const T*>(x.in) + b * x.in_b + n * x.in_n + me.chunk * 8;
      const T* dsrc = static_cast<const T*>(x.dy) + b * x.dy_b + n * x.dy_n + me.chunk * 8;
      T* dst = static_cast<T*>(x.out) + b * x.out_b + n * x.out_n + me.chunk * 8;
#pragma unroll 1
      for (int h0 = lo; h0 < hi; h0 += U) {
        Row8<T> rx[U], rd[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          rx[k] = rd[k] = Row8<T>{};
          if (live && h0 + k < hi) {
            rx[k] = load8(src + (h0 + k) * x.in_h);
            rd[k] = load8(dsrc + (h0 + k) * x.dy_h);
          }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          float v[8], d[8], o[8];
          unpack(rd[k], d);
          me.other(rd[k], d, o);
          unpack(rx[k], v);
          float ss = 0.f, sg = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            d[i] = fmaf(o[i], me.s[i], d[i] * me.c[i]);  // g
            ss = fmaf(v[i], v[i], ss);
            sg = fmaf(d[i] * w[i], v[i], sg);
          }
          ss = row_sum<L>(ss);
          sg = row_sum<L>(sg);
          const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
          const float q = r * r * (sg * inv_d);
          // A row outside the tensor adds nothing: its x is 0, but its r may be infinite (eps = 0).
          const bool row = live && h0 + k < hi;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (row) acc[t][i] = fmaf(d[i], v[i] * r, acc[t][i]);
            v[i] = r * fmaf(-v[i], q, d[i] * w[i]);
          }
          if (row) store8(dst + (h0 + k) * x.out_h, v);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) part[(me.lane_row * L + me.chunk) * 8 + i] = acc[t][i];
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kThreads) {
      float s = 0.f;
      for (int r = 0; r < ROWS; ++r) s += part[r * L * 8 + d];
      p.partial[((size_t)blockIdx.x * 2 + t) * p.D + d] = s;
    }
  }
}

// Sums the blocks' weight gradients: 32 channels of one tensor a block.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float* partial, int blocks, int D, float* dwq,
                                                                float* dwk) {
  __shared__ float s[32][33];
  const int d = blockIdx.x * 32 + threadIdx.x, t = blockIdx.y;
  float* dw = t ? dwk : dwq;
  if (!dw) return;
  float a = 0.f;
  if (d < D)
    for (int b = threadIdx.y; b < blocks; b += 32) a += partial[((size_t)b * 2 + t) * D + d];
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  float v = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int od = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && od < D) dw[od] = v;
}

int lanes_for(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Tiles, head groups and grid. A unit costs its heads' rows plus about three
// rows' worth of angles; of all group counts the one whose longest block is
// shortest is taken.
int plan_units(RopeParams& p, int num_sms, int per_sm) {
  const int rows = kThreads / lanes_for(p.D), heads = p.t[0].heads + p.t[1].heads;
  p.tiles = (p.N + rows - 1) / rows;
  const long long tiles = (long long)p.tiles * p.B, slots = (long long)num_sms * per_sm;
  long long best = -1;
  p.groups = 1;
  for (int g = 1; g <= heads; ++g) {
    const long long rounds = (tiles * g + slots - 1) / slots;
    const long long cost = rounds * (3 + (heads + g - 1) / g);
    if (best < 0 || cost < best) best = cost, p.groups = g;
  }
  p.units = tiles * p.groups;
  return (int)(p.units < slots ? p.units : slots);
}

template <typename T, int L, bool INTER>
cudaError_t launch_typed(const RopeParams& p, bool backward, int grid, cudaStream_t st) {
  constexpr int U = sizeof(T) == 4 ? 2 : 4;
  if (backward) norm_rope_backward_kernel<T, L, INTER, U / 2><<<grid, kThreads, 0, st>>>(p);
  else rope_kernel<T, L, INTER, U><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_lanes(const RopeParams& p, bool backward, int grid, cudaStream_t st) {
  switch (lanes_for(p.D) + (p.interleaved ? 1 : 0)) {
    case 4: return launch_typed<T, 4, false>(p, backward, grid, st);
    case 5: return launch_typed<T, 4, true>(p, backward, grid, st);
    case 8: return launch_typed<T, 8, false>(p, backward, grid, st);
    case 9: return launch_typed<T, 8, true>(p, backward, grid, st);
    case 16: return launch_typed<T, 16, false>(p, backward, grid, st);
    case 17: return launch_typed<T, 16, true>(p, backward, grid, st);
    case 32: return launch_typed<T, 32, false>(p, backward, grid, st);
    default: return launch_typed<T, 32, true>(p, backward, grid, st);
  }
}

cudaError_t launch_any(const RopeParams& p, int type, bool backward, int grid, cudaStream_t st) {
  if (type == 0) return launch_lanes<__nv_bfloat16>(p, backward, grid, st);
  if (type == 1) return launch_lanes<__half>(p, backward, grid, st);
  return launch_lanes<float>(p, backward, grid, st);
}

constexpr int kForwardPerSm = 3, kBackwardPerSm = 2;

}  // namespace

cudaError_t launch_rope(RopeParams p, int type, int num_sms, cudaStream_t st) {
  const int grid = plan_units(p, num_sms, kForwardPerSm);
  return launch_any(p, type, false, grid, st);
}

size_t norm_rope_partial_bytes(int D, int num_sms) { return (size_t)num_sms * kBackwardPerSm * 2 * D * sizeof(float); }

cudaError_t launch_norm_rope_backward(RopeParams p, int type, float* dwq, float* dwk, int num_sms, cudaStream_t st) {
  const int grid = plan_units(p, num_sms, kBackwardPerSm);
  cudaError_t e = launch_any(p, type, true, grid, st);
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  norm_weight_grad_kernel<<<dim3((p.D + 31) / 32, 2), dim3(32, 32), 0, st>>>(p.partial, grid, p.D, dwq, dwk);
  return cudaGetLastError();
}

}  // namespace vsa
