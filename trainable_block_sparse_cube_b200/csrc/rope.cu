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
// once. A whole position times the fraction of a turn that a pair makes for
// one, in 64 bits, keeps just the fraction of a turn in the low 64 bits of the
// product: within 2^-31 of a turn for positions up to 2^31, where fp32 would
// have lost 20 of its 24 bits at 10^6. The rest of an fp32 position, in 2^-32,
// adds its own product.
//
// Bound by HBM: a row is read once and written once (the norm's backward
// reads x and dy). A lane moves 8 channels, a power of two of lanes a row, and
// a thread keeps one (token, 8 channels) place for all heads of its unit, so
// an angle is computed once for 24 or 80 rows of it. Two heads at a time are
// worked on as packed pairs of fp32 (half the instructions: the norm is near
// the issue limit otherwise), while the rows of the next heads, tensors and
// units are on their way into shared memory (Feed: the norm's backward of
// 16,384 tokens x 24 heads of 128 in bf16 took 82 us with one step's rows ahead
// in registers, 62 with it). A unit is a tile of tokens by a group of heads;
// the grid holds the blocks that fit on the GPU and each strides over the
// units, the number of groups being the one whose longest block is shortest
// (plan_units). 61,440 tokens x 24 heads with the norm: 130 to 139 us, 0.84 to
// 0.90 of the copy rate; 76,800 x 80 backward: 546 us, 0.89.
//
// The weight gradients are summed per thread over its rows, per block through
// shared memory, and over the blocks by a second kernel, always in the same
// order: no atomics, the same bits every time.
#include <cuda_fp16.h>

#include <type_traits>

#include "launch.cuh"
#include "packed.cuh"
#include "sm100_ptx.cuh"
#include "vsa_common.cuh"

namespace vsa {

namespace {

constexpr int kThreads = 128;
constexpr int kBackwardStages = 4;
constexpr int kForwardPerSm = 4, kBackwardPerSm = 3;      // blocks of an SM
constexpr int kForwardAngles = 3, kBackwardAngles = 2;    // rows whose work an angle's equals, see plan_units

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
// fp32: whole 32-byte sectors where `wide` says that they are aligned.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8], bool) {
  store8(p, x);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&x)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

template <typename T>
__device__ __forceinline__ void unpack_pair(const Row8<T>& a, const Row8<T>& b, F2 (&x)[8]) {
  float u[8], v[8];
  unpack(a, u);
  unpack(b, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = pair2(u[i], v[i]);
}

// Sums over the L lanes of a row, of both heads and N values at once (their
// chains of shuffles run beside one another).
template <int L, int N>
__device__ __forceinline__ void row_sums(F2 (&v)[N]) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) {
    F2 w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float2 f = split2(v[k]);
      w[k] = pair2(__shfl_xor_sync(0xffffffffu, f.x, o), __shfl_xor_sync(0xffffffffu, f.y, o));
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = add2(v[k], w[k]);
  }
}

// A token's positions: the whole part as 32 low bits and what is above them,
// and, of an fp32 one, the rest in 2^-32.
struct Positions {
  uint32_t low[kRopeAxes], rest[kRopeAxes];
  int high[kRopeAxes];
  float bad[kRopeAxes];  // NaN for a position that is no number or not below 2^63 in size, else 0

  __device__ __forceinline__ void whole(int a, long long v) {
    low[a] = (uint32_t)v;
    high[a] = (int)(v >> 32);
  }
  __device__ __forceinline__ Positions(const RopeParams& p, int b, int n) {
    if (p.pos_kind == 0) {  // the raster grid's (t, h, w)
      const unsigned th = p.by_w(n), t = p.by_h(th);
      whole(0, (long long)t + p.origin[0]);
      whole(1, (long long)(th - t * p.H) + p.origin[1]);
      whole(2, (long long)(n - th * p.W) + p.origin[2]);
      whole(3, 0);
    } else {
      const long long o = (long long)b * p.pos_batch + (long long)n * p.axes;
#pragma unroll
      for (int a = 0; a < kRopeAxes; ++a) {
        const bool there = a < p.axes;
        if (p.pos_kind == 1) {
          whole(a, there ? static_cast<const int*>(p.pos)[o + a] : 0);
        } else {
          const float v = there ? static_cast<const float*>(p.pos)[o + a] : 0.f, f = floorf(v);
          whole(a, (long long)f);
          rest[a] = (uint32_t)((v - f) * 4294967296.f);
          bad[a] = fabsf(v) < 0x1p63f ? 0.f : __int_as_float(0x7fc00000);
        }
      }
    }
  }
  template <typename V>
  __device__ __forceinline__ static V pick(const V (&v)[kRopeAxes], int a) {
    return a == 0 ? v[0] : a == 1 ? v[1] : a == 2 ? v[2] : v[3];
  }
};

// Sine and cosine of a pair's angle. The nearest quarter of a turn is taken off
// and what is left, at most an eighth of a turn, goes into the Taylor
// polynomials (to x^9 and x^8: 2e-9 and 3e-8 at the ends).
__device__ __forceinline__ void pair_turn(const RopeParams& p, const RopePair& f, const Positions& pos, float* sn,
                                          float* cs) {
  const uint32_t lo = Positions::pick(pos.low, f.axis);
  uint32_t t = __umulhi(lo, f.lo) + lo * f.hi + (uint32_t)Positions::pick(pos.high, f.axis) * f.lo;
  if (p.pos_kind == 2) {
    const uint32_t rest = Positions::pick(pos.rest, f.axis);
    t += __umulhi(rest, f.hi) + rest * f.whole;
  }
  const int quarter = (int)((t + (1u << 29)) >> 30);
  float x = (float)(int)(t - ((uint32_t)quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  if (p.pos_kind == 2) x += Positions::pick(pos.bad, f.axis);
  const float x2 = x * x;
  const float sine = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
  const float cosine = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const float u = quarter & 1 ? cosine : sine, v = quarter & 1 ? sine : cosine;
  *sn = quarter & 2 ? -u : u;
  *cs = (quarter + 1) & 2 ? -v : v;
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

  // Coefficients for the token's positions. `back` turns the other way.
  __device__ __forceinline__ void angles(const RopeParams& p, const RopePair* pairs, const Positions& pos, bool back) {
    const float dir = back ? -1.f : 1.f;
    if (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = 1.f;
        s[2 * i] = s[2 * i + 1] = 0.f;
        if (turned >> (2 * i) & 1u) {
          float sn, cs;
          pair_turn(p, pairs[chunk * 4 + i], pos, &sn, &cs);
          c[2 * i] = c[2 * i + 1] = cs;
          s[2 * i] = -dir * sn;
          s[2 * i + 1] = dir * sn;
        }
      }
    } else {
      // the two chunks of a pair of halves need the same eight angles: each computes four
      const int first = (chunk * 8) % (p.rot > 0 ? p.rot / 2 : 1) + (sign < 0.f ? 0 : 4);
      float cs[4], sn[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (turned) pair_turn(p, pairs[first + i], pos, &sn[i], &cs[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float oc = __shfl_sync(0xffffffffu, cs[i], partner), os = __shfl_sync(0xffffffffu, sn[i], partner);
        c[i] = sign < 0.f ? cs[i] : oc;
        s[i] = sign * dir * (sign < 0.f ? sn[i] : os);
        c[i + 4] = sign < 0.f ? oc : cs[i];
        s[i + 4] = sign * dir * (sign < 0.f ? os : sn[i]);
      }
    }
  }

  // The other channel of each pair (0 where a channel is not rotated, so that
  // an infinity there meets no zero coefficient; `full`: all are rotated).
  __device__ __forceinline__ void other(const Row8<T>& a, const Row8<T>& b, const F2 (&x)[8], bool full,
                                        F2 (&xp)[8]) const {
    if (INTER) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xp[i] = x[i ^ 1];
    } else {
      Row8<T> u, v;
#pragma unroll
      for (int i = 0; i < Row8<T>::REGS; ++i) {
        u.r[i] = __shfl_sync(0xffffffffu, a.r[i], partner);
        v.r[i] = __shfl_sync(0xffffffffu, b.r[i], partner);
      }
      unpack_pair(u, v, xp);
    }
    if (!full) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!(turned >> i & 1u)) xp[i] = 0;
    }
  }
};

// The pairs from the launch parameters to shared memory.
__device__ __forceinline__ void stage_rotation(const RopeParams& p, RopePair* pairs) {
  for (int j = threadIdx.x; j < p.rot / 2; j += kThreads) pairs[j] = p.pairs[j];
  __syncthreads();
}

// Unit u: heads lo .. hi (those of q, then those of k), batch b, tile of tokens.
struct Unit {
  int b, tile, lo, hi;
  __device__ __forceinline__ Unit(const RopeParams& p, unsigned u) {
    const unsigned bt = p.by_groups(u), g = u - bt * p.groups, heads = p.t[0].heads + p.t[1].heads;
    b = (int)p.by_tiles(bt);
    tile = (int)(bt - (unsigned)b * p.tiles);
    lo = (int)p.by_groups(heads * g);
    hi = (int)p.by_groups(heads * (g + 1));
  }
  // Its heads of tensor t.
  __device__ __forceinline__ int first(const RopeParams& p, int t) const { return max(lo - (t ? p.t[0].heads : 0), 0); }
  __device__ __forceinline__ int last(const RopeParams& p, int t) const {
    return min(hi - (t ? p.t[0].heads : 0), p.t[t].heads);
  }
};

// The rows that a thread will need, in the order in which it will need them: U
// heads a step (zeros where there are fewer, or no such token), through all
// its units. Each step's 16-byte pieces go to the thread's own slots of a
// stage, so no barrier is needed; a stage is filled again one step after it
// was read. A thread's 8 fp32 channels are two pieces, and there the lanes of
// a row copy for one another, each two pieces L apart: neighbours' pieces are
// then neighbours in memory and in the row's slots, and no 32-byte sector is
// read twice. The
// common step is a handful of instructions: addresses are kept up by
// additions (products and checks for every row were half of all instructions).
template <typename T, int L, int U, bool DY, int STAGES>
struct Feed {
  static constexpr int PIECES = (int)sizeof(T) / 2;  // 16-byte pieces of 8 channels
  static constexpr int SLOTS = U * (DY ? 2 : 1) * PIECES;
  static constexpr uint32_t STAGE = SLOTS * kThreads * 16, END = STAGES * STAGE;
  uint32_t mine, in, out;  // shared address of the thread's first slot; offsets of the stages filled and read next
  uint32_t target[PIECES]; // where its copies go, for the first row of a stage
  int ahead;               // elements between its copies
  unsigned u;
  int t, left;             // heads left in the tensor's part of the unit
  const T *src, *dsrc;
  long long step, dstep;   // elements between heads
  uint32_t bytes[PIECES];  // 16, or 0 for a piece outside the tensor

  __device__ __forceinline__ void start(const RopeParams& p, const void* smem, int rows, int lane_row, int chunk) {
    mine = ptx::smem_u32(smem) + threadIdx.x * 16 * PIECES;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      target[i] = mine + (chunk + L * i - chunk * PIECES) * 16;
    }
    ahead = L * 4;
    in = out = 0;
    u = blockIdx.x;
    t = -1;
    left = 0;
    for (int i = 0; i < STAGES - 1; ++i) load(p, rows, lane_row, chunk);
  }

  // The next tensor or unit that has heads.
  __device__ __forceinline__ void open(const RopeParams& p, int rows, int lane_row, int chunk) {
    do {
      if (++t == 2) t = 0, u += gridDim.x;
      if (u >= p.units) return;
      const Unit w(p, u);
      const RopeTensor& x = p.t[t];
      const int lo = w.first(p, t), n = w.tile * rows + lane_row;
      left = w.last(p, t) - lo;
      const bool live = n < p.N && chunk * (16 / (int)sizeof(T)) < p.D;
      // what lies outside is not read, and keeps an address inside
      const long long at = lo, b = live ? w.b : 0, m = live ? n : 0, c = live ? chunk * (16 / (int)sizeof(T)) : 0;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) bytes[i] = live && (chunk + L * i) * (16 / (int)sizeof(T)) < p.D ? 16 : 0;
      src = static_cast<const T*>(x.in) + b * x.in_b + m * x.in_n + at * x.in_h + c;
      step = x.in_h;
      if (DY) {
        dsrc = static_cast<const T*>(x.dy) + b * x.dy_b + m * x.dy_n + at * x.dy_h + c;
        dstep = x.dy_h;
      }
    } while (left <= 0);
  }

  __device__ __forceinline__ static void copy(uint32_t dst, const T* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  }

  // Copies of the next step, one group (an empty one behind the last).
  __device__ __forceinline__ void load(const RopeParams& p, int rows, int lane_row, int chunk) {
    if (left <= 0 && u < p.units) open(p, rows, lane_row, chunk);
    if (u < p.units) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool there = k < left;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const uint32_t dst = target[i] + in + k * PIECES * kThreads * 16, n = there ? bytes[i] : 0;
          const int far = n ? i * ahead : 0;
          copy(dst, src + far, n);
          if (DY) copy(dst + U * PIECES * kThreads * 16, dsrc + far, n);
        }
        if (k + 1 < left) {  // the last head's address stays for copies of nothing: it is inside and aligned
          src += step;
          if (DY) dsrc += dstep;
        }
      }
      left -= U;
    }
    ptx::cp_async_commit();
    in = in + STAGE == END ? 0 : in + STAGE;
  }

  // The oldest step's rows have arrived.
  __device__ __forceinline__ void wait() {
    ptx::cp_async_wait<STAGES - 2>();
    if (PIECES > 1) __syncwarp();
  }
  __device__ __forceinline__ Row8<T> row(int k) const {
    Row8<T> v;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.r[4 * i]), "=r"(v.r[4 * i + 1]), "=r"(v.r[4 * i + 2]), "=r"(v.r[4 * i + 3])
                   : "r"(mine + out + k * PIECES * kThreads * 16 + i * 16)
                   : "memory");
    return v;
  }
  __device__ __forceinline__ void next() { out = out + STAGE == END ? 0 : out + STAGE; }
};

// U: heads worked on at a time, an even number.
template <typename T, int L, bool INTER, int U>
__global__ void __launch_bounds__(kThreads, kForwardPerSm) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int STAGES = 3;
  __shared__ RopePair pairs[kRopePairs];
  __shared__ uint4 ring[STAGES][Feed<T, L, U, false, STAGES>::SLOTS][kThreads];
  constexpr int ROWS = kThreads / L;
  Place<T, L, INTER> me;
  me.init(p.D, p.rot);
  Feed<T, L, U, false, STAGES> feed;
  feed.start(p, ring, ROWS, me.lane_row, me.chunk);
  stage_rotation(p, pairs);
  const float inv_d = 1.f / (float)p.D;
  const bool full = p.rot == p.D;
  for (unsigned u = blockIdx.x; u < p.units; u += gridDim.x) {
    const Unit w(p, u);
    const int n = w.tile * ROWS + me.lane_row;
    const bool live = n < p.N && me.in_row;
    const Positions pos(p, w.b, n < p.N ? n : 0);
    me.angles(p, pairs, pos, p.back != 0);
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const RopeTensor& x = p.t[t];
      const int lo = w.first(p, t), heads = w.last(p, t) - lo;
      if (heads <= 0) continue;
      T* dst = static_cast<T*>(x.out) + w.b * x.out_b + n * x.out_n + lo * x.out_h + me.chunk * 8;
      const long long step = x.out_h;
      // y_i = r (x_i A_i + x'_i B_i), the weight folded into A and B
      F2 A[8], B[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) A[i] = both(me.c[i]), B[i] = both(me.s[i]);
      if (x.w && me.in_row) {
        const int pc = INTER ? me.chunk : me.chunk + (me.partner - (int)(threadIdx.x & 31));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          A[i] = both(me.c[i] * x.w[me.chunk * 8 + i]);
          // a channel that is not rotated has no partner, whose weight may be no number
          if (me.turned >> i & 1u) B[i] = both(me.s[i] * x.w[pc * 8 + (INTER ? i ^ 1 : i)]);
        }
      }
#pragma unroll 1
      for (int h0 = 0; h0 < heads; h0 += U) {
        feed.wait();
        Row8<T> now[U];
#pragma unroll
        for (int k = 0; k < U; ++k) now[k] = feed.row(k);
        feed.next();
        feed.load(p, ROWS, me.lane_row, me.chunk);
        // A step of few heads leaves out the pairs that are not there.
        auto rows = [&](auto pairs_of) {
          constexpr int P = decltype(pairs_of)::value;
          F2 o[P][8], r[P];
#pragma unroll
          for (int k = 0; k < P; ++k) {
            F2 v[8];
            unpack_pair(now[2 * k], now[2 * k + 1], v);
            me.other(now[2 * k], now[2 * k + 1], v, full, o[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[k][i] = fma2(o[k][i], B[i], mul2(v[i], A[i]));
            if (p.norm) {
              r[k] = mul2(v[0], v[0]);
#pragma unroll
              for (int i = 1; i < 8; ++i) r[k] = fma2(v[i], v[i], r[k]);
            }
          }
          if (p.norm) {
            row_sums<L>(r);
#pragma unroll
            for (int k = 0; k < P; ++k) {
              const float2 m = split2(fma2(r[k], both(inv_d), both(p.eps)));
              r[k] = pair2(rsqrtf(m.x), rsqrtf(m.y));
#pragma unroll
              for (int i = 0; i < 8; ++i) o[k][i] = mul2(o[k][i], r[k]);
            }
          }
#pragma unroll
          for (int k = 0; k < 2 * P; ++k) {
            float a[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = k & 1 ? split2(o[k / 2][i]).y : split2(o[k / 2][i]).x;
            if (live && h0 + k < heads) store8(dst, a, p.wide != 0);
            dst += step;
          }
        };
        if (U > 2 && heads - h0 <= 2) rows(std::integral_constant<int, 1>());
        else rows(std::integral_constant<int, U / 2>());
      }
    }
  }
}

// Backward of the norm with the rotation: x.in = x, x.dy = dy, x.out = dx, the
// block's weight gradients to p.partial[block][tensor][D].
template <typename T, int L, bool INTER>
__global__ void __launch_bounds__(kThreads, kBackwardPerSm)
    norm_rope_backward_kernel(const __grid_constant__ RopeParams p) {
  constexpr int STAGES = kBackwardStages;
  extern __shared__ uint4 ring[];
  __shared__ RopePair pairs[kRopePairs];
  __shared__ float part[2][8][kThreads];  // a thread's sums of 8 channels over its rows so far
  constexpr int ROWS = kThreads / L;
  Place<T, L, INTER> me;
  me.init(p.D, p.rot);
  Feed<T, L, 2, true, STAGES> feed;
  ptx::let_next_start();
  feed.start(p, ring, ROWS, me.lane_row, me.chunk);
  stage_rotation(p, pairs);
  const float inv_d = 1.f / (float)p.D;
  const bool full = p.rot == p.D;
#pragma unroll
  for (int i = 0; i < 8; ++i) part[0][i][threadIdx.x] = part[1][i][threadIdx.x] = 0.f;
  for (unsigned u = blockIdx.x; u < p.units; u += gridDim.x) {
    const Unit w(p, u);
    const int n = w.tile * ROWS + me.lane_row;
    const bool live = n < p.N && me.in_row;
    const Positions pos(p, w.b, n < p.N ? n : 0);
    me.angles(p, pairs, pos, true);
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const RopeTensor& x = p.t[t];
      const int lo = w.first(p, t), heads = w.last(p, t) - lo;
      if (heads <= 0) continue;
      T* dst = static_cast<T*>(x.out) + w.b * x.out_b + n * x.out_n + lo * x.out_h + me.chunk * 8;
      const long long step = x.out_h;
      float wt[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) wt[i] = x.w && me.in_row ? x.w[me.chunk * 8 + i] : 1.f;
      F2 acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0;
#pragma unroll 1
      for (int h0 = 0; h0 < heads; h0 += 2) {
        F2 v[8], g[8], gw[8];
        const bool second = live && h0 + 1 < heads;
        feed.wait();
        {
          F2 d[8], o[8];
          const Row8<T> d0 = feed.row(2), d1 = feed.row(3);
          unpack_pair(feed.row(0), feed.row(1), v);
          feed.next();
          feed.load(p, ROWS, me.lane_row, me.chunk);
          unpack_pair(d0, d1, d);
          me.other(d0, d1, d, full, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = fma2(o[i], both(me.s[i]), mul2(d[i], both(me.c[i])));
        }
        F2 sum[2] = {0, 0};  // of x^2, of g w x
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          gw[i] = mul2(g[i], both(wt[i]));
          sum[0] = fma2(v[i], v[i], sum[0]);
          sum[1] = fma2(gw[i], v[i], sum[1]);
        }
        row_sums<L>(sum);
        const float2 m = split2(fma2(sum[0], both(inv_d), both(p.eps)));
        // A row outside the tensor adds nothing: its x is 0, but its r may be infinite (eps = 0).
        const F2 r = pair2(live ? rsqrtf(m.x) : 0.f, second ? rsqrtf(m.y) : 0.f);
        const F2 q = mul2(mul2(mul2(r, sum[1]), both(-inv_d)), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = mul2(v[i], r);
          acc[i] = fma2(g[i], v[i], acc[i]);
          v[i] = fma2(v[i], q, mul2(gw[i], r));
        }
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = split2(v[i]);
          a[i] = f.x, b[i] = f.y;
        }
        if (live) store8(dst, a, p.wide != 0);
        dst += step;
        if (second) store8(dst, b, p.wide != 0);
        dst += step;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = split2(acc[i]);
        part[t][i][threadIdx.x] += f.x + f.y;
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * p.D; e += kThreads) {
    const int t = e >= p.D, d = e - t * p.D;
    float s = 0.f;
    for (int r = 0; r < ROWS; ++r) s += part[t][d % 8][r * L + d / 8];
    p.partial[(size_t)blockIdx.x * 2 * p.D + e] = s;
  }
}

// Sums the blocks' weight gradients: 32 channels of one tensor a block.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float* partial, int blocks, int D, float* dwq,
                                                                float* dwk) {
  __shared__ float s[32][33];
  ptx::wait_for_previous();
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

// Tiles, head groups and grid. A unit costs its heads' rows plus `angles` rows'
// worth of work for its angles; of all group counts the one whose longest block
// is shortest is taken.
int plan_units(RopeParams& p, int num_sms, int per_sm, int angles) {
  const int rows = kThreads / lanes_for(p.D), heads = p.t[0].heads + p.t[1].heads;
  p.tiles = (p.N + rows - 1) / rows;
  const long long tiles = (long long)p.tiles * p.B, slots = (long long)num_sms * per_sm;
  long long best = -1;
  p.groups = 1;
  for (int g = 1; g <= heads && tiles * g < (1LL << 31) && heads * (g + 1LL) < (1LL << 31); ++g) {
    const long long rounds = (tiles * g + slots - 1) / slots;
    const long long cost = rounds * (angles + (heads + g - 1) / g);
    if (best < 0 || cost < best) best = cost, p.groups = g;
  }
  p.units = (unsigned)(tiles * p.groups);
  p.by_groups = Divisor(p.groups);
  p.by_tiles = Divisor(p.tiles);
  return (int)(p.units < slots ? p.units : slots);
}

template <typename T, int L, bool INTER>
cudaError_t launch_typed(const RopeParams& p, bool backward, int grid, cudaStream_t st) {
  constexpr int U = sizeof(T) == 4 ? 2 : 4;
  if (backward) {
    constexpr int smem = Feed<T, L, 2, true, kBackwardStages>::END;
    const cudaError_t e = allow_smem<norm_rope_backward_kernel<T, L, INTER>>(smem);
    if (e != cudaSuccess) return e;
    norm_rope_backward_kernel<T, L, INTER><<<grid, kThreads, smem, st>>>(p);
  } else rope_kernel<T, L, INTER, U><<<grid, kThreads, 0, st>>>(p);
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


}  // namespace

cudaError_t launch_rope(RopeParams p, int type, int num_sms, cudaStream_t st) {
  const int grid = plan_units(p, num_sms, kForwardPerSm, kForwardAngles);
  return launch_any(p, type, false, grid, st);
}

size_t norm_rope_partial_bytes(int D, int num_sms) { return (size_t)num_sms * kBackwardPerSm * 2 * D * sizeof(float); }

cudaError_t launch_norm_rope_backward(RopeParams p, int type, float* dwq, float* dwk, int num_sms, cudaStream_t st) {
  const int grid = plan_units(p, num_sms, kBackwardPerSm, kBackwardAngles);
  cudaError_t e = launch_any(p, type, true, grid, st);
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  return launch_behind(norm_weight_grad_kernel, dim3((p.D + 31) / 32, 2), dim3(32, 32), 0, st,
                       (const float*)p.partial, grid, p.D, dwq, dwk);
}

}  // namespace vsa
