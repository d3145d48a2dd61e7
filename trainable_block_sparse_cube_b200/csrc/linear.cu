// Linear product with its epilogue, and its gradients:
//
//   forward   y = act(x W^T + b) + res,  z = x W^T + b saved for the backward
//   backward  dz = dy act'(z);  dx = dz W,  dW = dz^T x,  db = sum over rows of dz
//
// x, y, res, z and their gradients are strided views [B, heads, N, D] read and
// written in place as B x N rows of heads * D channels, so the product takes
// the attention's output and makes its v without a copy.
//
// Three kernels make a product:
//  * gemm_kernel, tensor cores. A pair of CTAs computes a tile of 256 x bn:
//    each CTA holds 128 rows of A and half of B's rows, tcgen05.mma
//    (cta_group::2) reads both halves, so a CTA loads 16 + bn/16 KB a 64-long
//    step of the contraction instead of the 16 + bn/8 KB of a lone CTA: the
//    L2 -> SM rate, not the tensor cores, would bound the latter. Two warps
//    issue the loads (7 stages of 32 KB, or more and smaller ones), one the
//    MMAs, eight the epilogue of the tile before (two accumulators of up to 256
//    columns fill the SM's tensor memory). Bound by the tensor cores where the
//    product is large.
//  * finish_kernel joins the parts of a contraction that was split because it
//    has too few tiles for 74 pairs, always in the same order.
//  * few_rows_kernel, up to 32 rows: W straight from memory into warp-wide
//    MMAs. One pass over W is its floor; it is bound by the latency of that
//    pass (2 rows of 1536 -> 9216: 10.9 us alone, 4.4 at the copy rate, memory
//    32% busy).
//
// Sums are fp32; the result is rounded once. dz is rounded to the operands'
// type before its products, as the tensor cores read it; db is summed from
// the unrounded values.
#include <cuda_fp16.h>

#include <type_traits>

#include "launch.cuh"
#include "pair_ptx.cuh"
#include "vsa_common.cuh"

namespace vsa {

namespace {

using namespace ptx;

// How many warps gave up waiting, in the products of each stream that has a
// word here. They only grow: a reader compares with what it saw before, so
// that none can take a failure from another, and none is lost between a look
// and a reset.
__device__ unsigned g_linear_failures[kLinearFailureWords];

constexpr int kRingBytes = 7 * 32768, kTileA = 16384;
constexpr int kEpiWarps = 8, kThreads = 96 + 32 * kEpiWarps;  // two warps load, one issues MMAs
constexpr int kAccColumns = 256;

struct Barriers {
  uint64_t full[kGemmMaxStages], empty[kGemmMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drained;
  uint32_t tmem;
  uint32_t stop;  // the loads stop before this step, counted over the pair's units; see Waiter::stage
};
constexpr int kGemmSmem = 1024 + kRingBytes + (int)sizeof(Barriers);
static_assert(kGemmSmem <= 227 * 1024, "shared memory");

// ---------------------------------------------------------------- arithmetic
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// Two z held within what their slopes can take: these are 0 and 1 long before
// 1e9, whose cube is finite. Far out, and at the infinity that a sum becomes
// when it is rounded to fp16, z would meet factors of 0. A NaN stays one. (Held
// before they are unpacked: as floats it took 4% of dz's time.)
template <typename T>
__device__ __forceinline__ uint32_t finite2(uint32_t v);
template <>
__device__ __forceinline__ uint32_t finite2<__nv_bfloat16>(uint32_t v) {
  const __nv_bfloat162 most = __float2bfloat162_rn(1e9f), z = *reinterpret_cast<const __nv_bfloat162*>(&v);
  const __nv_bfloat162 r = __hmax2_nan(__hmin2_nan(z, most), __hneg2(most));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t finite2<__half>(uint32_t v) {
  const __half2 most = __float2half2_rn(65504.f), z = *reinterpret_cast<const __half2*>(&v);
  const __half2 r = __hmax2_nan(__hmin2_nan(z, most), __hneg2(most));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<T>(r[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// z s(v) and its slope s + z s (1 - s) v' are silu (v = z) and the tanh form
// of gelu (v = 2 sqrt(2/pi) (z + 0.044715 z^3)); both keep their relative
// accuracy where z is far below 0.
constexpr float kTanhA = 1.5957691216057308f, kTanhB = 0.07135481282805f;  // 2 sqrt(2/pi), that times 0.044715

// The hardware's 2^x and 1/x; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid(float v) { return rcp_approx(1.f + exp2_approx(-kLog2e * v)); }

// gelu is z P(z) with the normal distribution function P. Its tail
// h = P(-|z|) = exp(-z^2 / 2) t q(t) with t = 1 / (1 + 0.3111 |z|), in the form
// of Hastings' approximations: q is of degree 7, fitted for this to the least
// relative error over |z| <= 20 (1.9e-7). In fp32 the rounding of the exponent
// adds to that with z^2: 5e-7 up to |z| = 1, 8e-7 up to 4, 4e-6 up to 9 and
// 7.5e-6 up to 13; beyond 13.2 the exponential is below 2^-126 and h is 0. All
// of it is far below the results' half step, at a quarter of the instructions
// of the complementary error function (16384 x 1536 -> 6144: 222 us, with
// erfcf 399).
__device__ __forceinline__ float normal_tail(float a, float* density) {
  const float t = rcp_approx(fmaf(0.3111269772052765f, a, 1.f));
  const float e = exp2_approx(-0.5f * kLog2e * (a * a));
  float q = 0.03574991226196289f;
  q = fmaf(q, t, -0.13957644999027252f);
  q = fmaf(q, t, 0.14943377673625946f);
  q = fmaf(q, t, -0.011147385463118553f);
  q = fmaf(q, t, 0.10849696397781372f);
  q = fmaf(q, t, 0.10846728086471558f);
  q = fmaf(q, t, 0.12446772307157516f);
  q = fmaf(q, t, 0.12410826236009598f);
  *density = e;
  return q * t * e;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == kActSilu) return z * sigmoid(z);
  if (ACT == kActGeluTanh) return z * sigmoid(z * fmaf(kTanhB, z * z, kTanhA));
  if (ACT == kActGelu) {
    float e;
    const float a = fminf(fabsf(z), 20.f);  // the tail is 0 beyond: an infinite z meets no 0 x infinity
    return fmaf(-a, normal_tail(a, &e), z < 0.f ? 0.f : z);
  }
  return z;
}

// z is finite or NaN, and its square finite; see finite2.
template <int ACT>
__device__ __forceinline__ float slope(float z) {
  if (ACT == kActSilu) {
    const float s = sigmoid(z);
    return fmaf(z, fmaf(-s, s, s), s);
  }
  if (ACT == kActGeluTanh) {
    const float s = sigmoid(z * fmaf(kTanhB, z * z, kTanhA));
    return fmaf(z * fmaf(3.f * kTanhB, z * z, kTanhA), fmaf(-s, s, s), s);
  }
  if (ACT == kActGelu) {  // P(z) + z exp(-z^2 / 2) / sqrt(2 pi)
    float e;
    const float h = normal_tail(fminf(fabsf(z), 20.f), &e);
    return fmaf(0.3989422804014327f * z, e, z < 0.f ? h : 1.f - h);
  }
  return 1.f;
}

// One branch for all N values, whose chains of exponential and reciprocal then
// run beside one another.
template <int ACT, int N>
__device__ __forceinline__ void activate_all(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = activate<ACT>(v[i]);
}
template <int N>
__device__ __forceinline__ void activate_n(float (&v)[N], int act) {
  if (act == kActSilu) activate_all<kActSilu>(v);
  else if (act == kActGelu) activate_all<kActGelu>(v);
  else if (act == kActGeluTanh) activate_all<kActGeluTanh>(v);
}
template <int ACT, int N>
__device__ __forceinline__ void times_slope_all(float (&v)[N], const float (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= slope<ACT>(z[i]);
}
template <int N>
__device__ __forceinline__ void times_slope(float (&v)[N], const float (&z)[N], int act) {
  if (act == kActSilu) times_slope_all<kActSilu>(v, z);
  else if (act == kActGelu) times_slope_all<kActGelu>(v, z);
  else if (act == kActGeluTanh) times_slope_all<kActGeluTanh>(v, z);
}

__device__ __forceinline__ void add_bias8(float (&v)[8], const float* bias) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(bias)), b = __ldg(reinterpret_cast<const float4*>(bias) + 1);
  v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
  v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
}

template <typename T>
__device__ __forceinline__ void pack16(const float (&v)[16], uint32_t (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
}

// 32 bytes, in one access where `wide` says that they are aligned to it; only
// the first 16 unless `both`.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8], bool wide, bool both) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    if (both) static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void load32(const void* p, uint32_t (&v)[8], bool wide, bool both) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0];
    const uint4 b = both ? static_cast<const uint4*>(p)[1] : make_uint4(0, 0, 0, 0);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// Asked for here and not where it is used.
__device__ __forceinline__ float4 load_bias(const float* p) {
  float4 v;
  asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

template <typename T>
__device__ __forceinline__ T* view_at(const RowsView& v, int b, int head, int n) {
  return static_cast<T*>(v.data) + b * v.s_b + head * v.s_h + n * v.s_n;
}
template <typename T>
__device__ __forceinline__ T* at(const RowsView& v, int b, int n, int c) {
  return static_cast<T*>(v.data) + b * v.s_b + (c / v.D) * v.s_h + n * v.s_n + c % v.D;
}

// ---------------------------------------------------------------- tensor cores
// Limit of the waits for what is under way already: loads and MMAs that were issued.
constexpr unsigned long long kDrainNs = 2000000000ull;

// Bounded waits; a warp's lanes give up together.
struct Waiter {
  unsigned long long limit;
  unsigned word;  // of g_linear_failures
  // A loading warp's wait for a stage. While the pair's MMAs go on, the only
  // other end is `stop`: the warp that issues them, whose waits have the limit,
  // gives up at some step m and sets it to m + stages in both CTAs. The steps
  // before that need nothing but MMAs that are under way, so both CTAs issue
  // their loads of exactly these steps, for which that warp then waits: no
  // load is in flight when the pair's shared memory goes. The time here is
  // above all that the other warps may wait in between, and runs out in no
  // other case.
  __device__ __forceinline__ bool stage(uint64_t* bar, uint32_t parity, const uint32_t* stop, uint32_t step) const {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || stage_loop(bar, parity, stop, step);
  }
  // Out of line: the code that every launch fetches anew stays short.
  __device__ __noinline__ bool stage_loop(uint64_t* bar, uint32_t parity, const uint32_t* stop, uint32_t step) const {
    uint64_t t0 = 0;
    for (int late = 0;;) {
      bool done = false;
#pragma unroll 1
      for (int i = 0; i < 64 && !done; ++i) done = mbar_try_wait(bar, parity);
      if (__all_sync(0xffffffffu, done)) return true;
      if (__any_sync(0xffffffffu, step >= load_cluster(stop))) return false;
      const uint64_t now = globaltimer_ns();
      if (!t0) t0 = now;
      late += now - t0 > 8 * limit + kDrainNs;
      if (__any_sync(0xffffffffu, late > 4096)) return gave_up();
    }
  }
  // `seen`: what an earlier look at the barrier found.
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity, bool seen = false) const {
    return __all_sync(0xffffffffu, seen) || __all_sync(0xffffffffu, mbar_wait(bar, parity, limit)) || gave_up();
  }
  __device__ __forceinline__ bool pair(uint64_t* bar, uint32_t parity) const {  // arrivals of both CTAs
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, limit)) || gave_up();
  }
  __device__ __forceinline__ bool gave_up() const {
    atomicAdd(&g_linear_failures[word], 1u);
    return false;
  }
};

// Tiles in the order they run in. The pairs that run together take a block of
// kTileGroup row tiles by the columns beside it, so that what they load from L2 is
// few rows of A and few of B (8192^3: 2.25 -> 1.10 GB from DRAM).
// Every second block goes back over the columns, whose last rows of B are still
// in L2 (16384 x 5120 x 5120 with a residual 952 -> 801 MB; 76800 rows of it,
// which the power cap slows, 3282-3409 -> 3136-3244 us).
__device__ __forceinline__ void tile_place(const TileOrder& o, int tile, int* rt, int* ct) {
  const int group = (int)o.by_block(tile), in = tile - group * o.block;
  const int high = min(kTileGroup, o.rows - group * kTileGroup);
  const int col = high == kTileGroup ? in / kTileGroup : in / high;
  *rt = group * kTileGroup + in - col * high;
  *ct = group & 1 ? o.cols - 1 - col : col;
}

// A work unit: a tile, or one part of the contraction of a tile of the last
// round, which has too few tiles for all pairs.
struct Unit {
  int batch, row0, col0, part, k0, k1;  // part: index of the partial tile, -1 for a whole contraction
  __device__ __forceinline__ Unit(const GemmParams& p, unsigned u) {
    unsigned t = u;
    part = -1;
    steps(p, u, &k0, &k1);
    if (u >= p.whole) {
      part = u - p.whole;
      t = p.whole + part - (int)p.by_rest(part) * p.rest;
    }
    int rt, ct;
    tile_place(p.order, t, &rt, &ct);
    batch = p.batches > 1 ? (int)p.by_row_tiles(rt) : 0;
    row0 = (rt - batch * p.row_tiles) * 256;
    col0 = ct * p.bn;
  }
  __device__ __forceinline__ static void steps(const GemmParams& p, unsigned u, int* k0, int* k1) {
    *k0 = 0;
    *k1 = p.kblocks;
    if (u >= p.whole) {
      const unsigned split = p.by_rest(u - p.whole);
      *k0 = (int)((unsigned)p.kblocks * split / p.splits);
      *k1 = (int)((unsigned)p.kblocks * (split + 1) / p.splits);
    }
  }
};

// Stage of the ring and the parity of its use.
struct Ring {
  int stage = 0, stages;
  uint32_t parity = 0;
  __device__ __forceinline__ explicit Ring(const GemmParams& p) : stages(p.stages) {}
  __device__ __forceinline__ void next() {
    if (++stage == stages) stage = 0, parity ^= 1;
  }
  __device__ __forceinline__ Ring after(int n) const {
    Ring r = *this;
    for (int i = 0; i < n; ++i) r.next();
    return r;
  }
};

// The end of the warp that issues the MMAs, when it gives up at `step`: the
// loads that both CTAs issue up to `stop` land. Out of line, as it hardly runs.
__device__ __noinline__ void give_up(const GemmParams& p, Barriers& sh, Ring ring, uint32_t step) {
  const int lane = threadIdx.x & 31;
  if (lane < 2) store_cluster(mapa(smem_u32(&sh.stop), lane), step + p.stages);
  uint32_t all = 0;
  for (unsigned u = blockIdx.x >> 1; u < (unsigned)p.units; u += gridDim.x >> 1) {
    int k0, k1;
    Unit::steps(p, u, &k0, &k1);
    all += k1 - k0;
  }
  const uint32_t end = min(all, step + p.stages);
  for (; p.stall != kStallUnloaded && step < end; ++step, ring.next())
    if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[ring.stage], ring.parity, kDrainNs))) break;
}

// KIND kGemmForward: A and B K-major. kGemmInput: A K-major, B MN-major.
// kGemmWeight: both MN-major, the contraction running over batches of rows.
template <int KIND, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ GemmParams p) {
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  Barriers& sh = *reinterpret_cast<Barriers*>(raw + (base - smem_u32(raw)) + kRingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const unsigned pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, units = (unsigned)p.units;
  const int half = p.bn / 2;  // rows of B in a CTA
  const Waiter wait{p.wait_ns, p.failures};

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&sh.full[s], 1), mbar_init(&sh.empty[s], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.acc_full[i], 1), mbar_init(&sh.acc_empty[i], 2 * kEpiWarps);
    mbar_init(&sh.drained, 1);
    sh.stop = ~0u;
    fence_mbar_init();
    prefetch_tmap(&p.ta);
    prefetch_tmap(&p.tb);
  }
  if (warp == 2) {
    tmem_alloc_pair(&sh.tmem, 512);
    tmem_relinquish_pair();
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  ptx::wait_for_previous();
  ptx::let_next_start();

  // The issuing warps run their loops as whole warps, so that what they
  // compute is uniform, and elect a lane to issue.
  if (warp < 2) {
    // ---- loads of this CTA's operand rows; both CTAs' complete on the even
    // CTA's barriers. The two warps take every second step.
    const int b_boxes = (half + 63) / 64;
    const uint32_t b_bytes = KIND == kGemmForward ? half * 128 : b_boxes * 8192;
    const uint32_t full0 = mapa(smem_u32(&sh.full[0]), 0);
    const bool load = p.stall != kStallUnloaded;
    Ring ring(p);
    // A look at the next barrier is taken before this step's work: its answer
    // is there when it is needed.
    bool ok = true, mine = warp == 0, seen = true;
    uint32_t step = 0;  // of all units
    for (unsigned u = pair; ok && u < units; u += pairs) {
      // Divisions here; the steps keep their coordinates up by additions (a
      // division costs the issuing warp more than a load).
      const Unit w(p, u);
      const int row = w.row0 + (int)rank * 128, col = w.col0 + (int)rank * half;
      int ch0, ch1, cc0, cc1, bh0, bh1, bc0, bc1;  // kGemmWeight: head and channel of A's and B's boxes
      int k, kh, kend;                             // channel and head of the step, or row and batch of rows
      if (KIND == kGemmWeight) {
        ch0 = row / p.a_d, cc0 = row - ch0 * p.a_d;
        ch1 = (row + 64) / p.a_d, cc1 = row + 64 - ch1 * p.a_d;
        bh0 = col / p.b_d, bc0 = col - bh0 * p.b_d;
        bh1 = (col + 64) / p.b_d, bc1 = col + 64 - bh1 * p.b_d;
        kh = w.k0 / p.kblocks_batch;
        k = (w.k0 - kh * p.kblocks_batch) * 64;
        kend = p.kblocks_batch * 64;
      } else {
        kh = w.k0 * 64 / p.a_d;
        k = w.k0 * 64 - kh * p.a_d;
        kend = p.a_d;
      }
      // What a CTA whose rows lie behind the last computes is not stored: it
      // loads none, and a few rows are loaded as a smaller box (boxes of 128
      // rows with fewer than 16 of them inside the tensor are slow: the input's
      // gradient of 9 x 4096 x 4096 25.4 -> 17.5 us).
      const bool load_a = KIND == kGemmWeight || row < p.rows;
      const uint32_t a_bytes = KIND == kGemmWeight ? kTileA : p.a_rows * 128;
      const uint32_t pair_bytes = 2 * b_bytes + (KIND == kGemmWeight || w.row0 + 128 < p.rows ? 2 : 1) * a_bytes;
      for (int kb = w.k0; kb < w.k1; ++kb, ++step, ring.next()) {
        const int s = ring.stage;
        // passes at once where no use came before
        if (mine) {
          ok = __all_sync(0xffffffffu, seen) || wait.stage(&sh.empty[s], ring.parity ^ 1, &sh.stop, step);
          if (!ok) break;
          const Ring next = ring.after(2);
          seen = mbar_test(&sh.empty[next.stage], next.parity ^ 1);
          if (p.stall == kStallLate && rank == 1 && step < 2) {  // test hook: until the MMAs are given up, or about 1 s
            for (int i = 0; i < 1000000 && load_cluster(&sh.stop) == ~0u; ++i) __nanosleep(1000);
            __syncwarp();
          }
        }
        if (mine && elect_one()) {
          const uint32_t bar = full0 + s * 8;
          const uint32_t a = base + s * p.stage_bytes, b = a + p.tile_a;
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], pair_bytes);
          if (load) {
            if (KIND == kGemmWeight) {
              tma_load_4d_pair(a, &p.ta, bar, cc0, k, ch0, kh);
              tma_load_4d_pair(b, &p.tb, bar, bc0, k, bh0, kh);
              tma_load_4d_pair(a + 8192, &p.ta, bar, cc1, k, ch1, kh);
              if (b_boxes > 1) tma_load_4d_pair(b + 8192, &p.tb, bar, bc1, k, bh1, kh);
            } else {
              if (load_a) tma_load_4d_pair(a, &p.ta, bar, k, row, kh, w.batch);
              if (KIND == kGemmForward) {
                tma_load_4d_pair(b, &p.tb, bar, kb * 64, col, 0, 0);
              } else {
                tma_load_4d_pair(b, &p.tb, bar, col, kb * 64, 0, 0);
                if (b_boxes > 1) tma_load_4d_pair(b + 8192, &p.tb, bar, col + 64, kb * 64, 0, 0);
              }
            }
          }
        }
        mine = !mine;
        k += 64;
        if (k >= kend) k = 0, ++kh;
      }
    }
    // The MMAs' last arrivals on these barriers come before the shared memory
    // goes; stages that no step used have none.
    if (ok && warp == 0) {
      const int used = min(p.stages, (int)step);
      for (int i = used; i < p.stages; ++i) ring.next();
      for (int i = 0; ok && i < used; ++i, ring.next())
        ok = wait.stage(&sh.empty[ring.stage], ring.parity ^ 1, &sh.stop, step + p.stages - used + i);
    }
  } else if (warp == 2) {
    if (rank == 0) {
      // ---- MMAs of the pair
      const uint32_t idesc =
          idesc_f16_f32(256, p.bn, KIND == kGemmWeight, KIND != kGemmForward, std::is_same<T, __nv_bfloat16>::value);
      constexpr uint32_t A_STEP = (KIND == kGemmWeight ? 2048 : 32) >> 4;
      constexpr uint32_t B_STEP = (KIND == kGemmForward ? 32 : 2048) >> 4;
      const uint64_t ad0 = sdesc_sw128(base, KIND == kGemmWeight ? 8192 : 16, 1024);
      const uint64_t bd0 = sdesc_sw128(base + p.tile_a, KIND == kGemmForward ? 16 : 8192, 1024);
      Ring ring(p);
      int tile = 0;
      uint32_t step = 0;  // of all units
      bool ok = true, seen = false;
      for (unsigned u = pair; ok && u < units; u += pairs, ++tile) {
        int k0, k1;
        Unit::steps(p, u, &k0, &k1);
        const int buf = tile & 1, use = tile >> 1;
        const uint32_t acc = tmem + buf * kAccColumns;
        ok = !use || wait.pair(&sh.acc_empty[buf], (use - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t add = 0;
        for (int kb = k0; kb < k1; ++kb, ++step, ring.next()) {
          const int s = ring.stage;
          ok = wait.warp(&sh.full[s], ring.parity, seen);
          if (!ok) break;
          tc_fence_after();
          const Ring next = ring.after(1);
          seen = mbar_test(&sh.full[next.stage], next.parity);
          if (elect_one()) {
            const uint64_t at = (uint64_t)(s * (p.stage_bytes >> 4)), ad = ad0 + at, bd = bd0 + at;
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_f16_ss_pair(acc, ad + i * A_STEP, bd + i * B_STEP, idesc, i ? 1u : add);
            mma_commit_pair(&sh.empty[s]);
            if (kb + 1 == k1) mma_commit_pair(&sh.acc_full[buf]);
          }
          add = 1;
        }
      }
      if (!ok) give_up(p, sh, ring, step);
      // The MMAs end before the tensor memory goes, also where an epilogue gave up on them.
      if (elect_one()) mma_commit_pair(&sh.drained);
      mbar_wait(&sh.drained, 0, kDrainNs);
    }
  } else {
    // ---- epilogue: a warp takes 32 rows, a row a lane, and one half of the tile's
    // columns, 32 at a time, from tensor memory straight to global memory in
    // whole 32-byte sectors. Shared memory has no bandwidth to spare: the MMAs
    // read 64 bytes a cycle of it and the loads write as many (staged there and
    // stored by TMA, 16384 x 1536 x 6144 took 299 thousand cycles, with
    // gelu_tanh 342; straight, 292 and 297).
    const int quarter = warp & 3, groups = p.bn / 32;
    const int g0 = warp < 7 ? 0 : (groups + 1) / 2, g1 = warp < 7 ? (groups + 1) / 2 : groups;
    const bool plain = !p.bias && !p.z.data && !p.residual.data && p.act == kActNone, wide = p.wide != 0;
    int tile = 0;
    for (unsigned u = pair; u < units; u += pairs, ++tile) {
      const Unit w(p, u);
      const int buf = tile & 1;
      const int in_tile = (int)rank * 128 + quarter * 32 + lane, n = w.row0 + in_tile;
      const bool live = n < p.rows, some = n - lane < p.rows;
      const uint32_t acc0 = tmem_addr(tmem, quarter * 32, buf * kAccColumns);
      T* const out = view_at<T>(p.out, w.batch, 0, n);
      // The bias and the residual of a group are asked for one group ahead, of
      // the first one before the tile is there.
      const bool more = p.bias || p.residual.data;
      float4 bias[8];
      uint32_t res[2][8];
      auto ask = [&](int g) {
        const int col = w.col0 + g * 32, left = p.F - col;
        if (!some || g >= g1 || left <= 0) return;
        if (p.bias) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (4 * i < left) bias[i] = load_bias(p.bias + col + 4 * i);
        }
        if (p.residual.data && live) {
          const int head = p.out.heads > 1 ? col / p.out.D : 0;
          const T* const src = view_at<T>(p.residual, w.batch, head, n) + (col - head * p.out.D);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (16 * j < left) load32(src + 16 * j, res[j], wide, left > 16 * j + 8);
        }
      };
      if (more && w.part < 0) ask(g0);
      if (!wait.warp(&sh.acc_full[buf], (tile >> 1) & 1)) break;
      tc_fence_after();
      if (w.part >= 0) {  // a part of the contraction: fp32 sums
        float* const dst = p.partial + ((long long)w.part * 256 + in_tile) * p.bn;
#pragma unroll 1
        for (int g = g0; g < g1 && some && w.col0 + g * 32 < p.F; ++g) {
          uint32_t r[32];
          tmem_ld32(acc0 + g * 32, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v[8] = {r[8 * j],     r[8 * j + 1], r[8 * j + 2], r[8 * j + 3],
                                   r[8 * j + 4], r[8 * j + 5], r[8 * j + 6], r[8 * j + 7]};
            if (live) store32(dst + g * 32 + 8 * j, v, wide, true);
          }
        }
      } else if (plain) {
#pragma unroll 1
        for (int g = g0; g < g1; g += 2) {
          const int col = w.col0 + g * 32, left = p.F - col;  // columns up to the edge, a multiple of 8
          if (!some || left <= 0) break;
          const bool two = g + 1 < g1;
          uint32_t r[64];
          tmem_ld32(acc0 + g * 32, reinterpret_cast<uint32_t (&)[32]>(r[0]));
          if (two) tmem_ld32(acc0 + g * 32 + 32, reinterpret_cast<uint32_t (&)[32]>(r[32]));
          tmem_wait_ld();
          const int head = p.out.heads > 1 ? col / p.out.D : 0;
          T* const dst = out + head * p.out.s_h + (col - head * p.out.D);
          // a second group lies in the next head only where heads are 64 wide and the first is their second half
          const bool turn = two && p.out.heads > 1 && (col + 32) % p.out.D == 0;
          T* const dst2 = turn ? out + (head + 1) * p.out.s_h : dst + 32;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((j < 2 || two) && 16 * j < left) {
              float v[16];
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[16 * j + i]);
              pack16<T>(v, o);
              if (live) store32(j < 2 ? dst + 16 * j : dst2 + 16 * (j - 2), o, wide, left > 16 * j + 8);
            }
          }
        }
      } else {
#pragma unroll 1
        for (int g = g0; g < g1; ++g) {
          const int col = w.col0 + g * 32, left = p.F - col;
          if (!some || left <= 0) break;
          uint32_t r[32];
          tmem_ld32(acc0 + g * 32, r);
          const int head = p.out.heads > 1 ? col / p.out.D : 0, ch = col - head * p.out.D;
          tmem_wait_ld();
          float v[2][16];
          uint32_t x[2][8];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i / 16][i % 16] = __uint_as_float(r[i]);
          if (p.bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* const q = &v[i / 4][i % 4 * 4];
              q[0] += bias[i].x, q[1] += bias[i].y, q[2] += bias[i].z, q[3] += bias[i].w;
            }
          }
          if (p.residual.data) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i / 8][i % 8] = res[i / 8][i % 8];
          }
          if (more) ask(g + 1);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (16 * j >= left) break;
            const bool both = left > 16 * j + 8;
            uint32_t o[8];
            if (p.z.data) {
              pack16<T>(v[j], o);
              if (live) store32(view_at<T>(p.z, w.batch, head, n) + ch + 16 * j, o, wide, both);
            }
            activate_n(v[j], p.act);
            if (p.residual.data) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 f = unpack2<T>(x[j][i]);
                v[j][2 * i] += f.x;
                v[j][2 * i + 1] += f.y;
              }
            }
            pack16<T>(v[j], o);
            if (live) store32(out + head * p.out.s_h + ch + 16 * j, o, wide, both);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&sh.acc_empty[buf]), 0));
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 2) {
    if (rank) mbar_wait(&sh.drained, 0, kDrainNs);  // committed before the barrier above
    __syncwarp();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- split contractions
// out = act(sum of the parts + bias) + residual of the split tiles, 8 columns a thread.
template <typename T>
__global__ void __launch_bounds__(256) finish_kernel(const FinishParams p) {
  ptx::wait_for_previous();
  const int groups = p.bn / 8, per_tile = 256 * groups;
  const int tile = blockIdx.x / (per_tile / 256), in = (blockIdx.x % (per_tile / 256)) * 256 + threadIdx.x;
  int rt, ct;
  tile_place(p.order, p.first + tile, &rt, &ct);
  const int b = rt / p.row_tiles, r = in / groups, cc = (in - r * groups) * 8;
  const int n = (rt - b * p.row_tiles) * 256 + r, c = ct * p.bn + cc;
  if (n >= p.rows || c >= p.F) return;
  const float* src = p.partial + ((long long)tile * 256 + r) * p.bn + cc;
  const long long part = (long long)p.rest * 256 * p.bn;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float4 x = __ldcs(reinterpret_cast<const float4*>(src + s * part));
    const float4 y = __ldcs(reinterpret_cast<const float4*>(src + s * part) + 1);
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
  }
  if (p.bias) add_bias8(v, p.bias + c);
  if (p.z.data) *reinterpret_cast<uint4*>(at<T>(p.z, b, n, c)) = pack8<T>(v);
  activate_n(v, p.act);
  if (p.residual.data) {
    float x[8];
    unpack8<T>(*reinterpret_cast<const uint4*>(at<T>(p.residual, b, n, c)), x);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += x[k];
  }
  *reinterpret_cast<uint4*>(at<T>(p.out, b, n, c)) = pack8<T>(v);
}

// ---------------------------------------------------------------- few rows
constexpr int kFewColumns = 16;

// D += A B with A [16 x 16] (W's rows), B [16 x 8] (x's rows as columns).
template <typename T>
__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 * NT >= batches * rows rows; a block computes 16 columns of all of them,
// its warps' shares of the contraction joined in shared memory, in order. W is
// read once, straight into the fragments of a warp-wide MMA: the order of the
// contraction does not matter as long as W and x agree, so a lane takes 8
// channels in a row of two of W's rows and of one row of x, which are its
// places in two MMAs of 16 channels. Bound by the latency of W's loads, of
// which a warp has two to four in flight; there is no arithmetic to speak of
// (with products and sums on the ordinary pipes eight rows took three times as
// long as one).
template <int NT, int WARPS, typename T>
__global__ void __launch_bounds__(32 * WARPS) few_rows_kernel(const FewRowsParams p) {
  constexpr int UNROLL = NT > 2 ? 2 : 4;
  __shared__ float part[WARPS][NT][kFewColumns][8 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int M = p.batches * p.rows, f0 = blockIdx.x * kFewColumns;
  const T* const w0 = static_cast<const T*>(p.w) + (long long)(f0 + g) * p.w_stride;
  const bool low = f0 + g + 8 < p.F;  // F is a multiple of 8: the upper eight rows are there, the lower may not be
  const T* const w1 = low ? w0 + 8 * p.w_stride : w0;
  const T* x[NT];
  bool there[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int m = 8 * i + g;
    there[i] = m < M;
    x[i] = there[i] ? at<T>(p.x, m / p.rows, m % p.rows, 0) : static_cast<const T*>(p.x.data);
  }
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const int steps = (p.K + 31) / 32, s0 = steps * warp / WARPS, s1 = steps * (warp + 1) / WARPS;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // the head that a step's channels lie in, kept up by additions
  int head = p.x.heads > 1 ? s0 * 32 / p.x.D : 0;
  int c = s0 * 32 - head * p.x.D + 8 * t;
#pragma unroll UNROLL
  for (int s = s0; s < s1; ++s) {
    const int k = s * 32 + 8 * t;
    uint4 a0 = zero, a1 = zero, b[NT];
    if (k < p.K) {
      a0 = __ldg(reinterpret_cast<const uint4*>(w0 + k));
      a1 = __ldg(reinterpret_cast<const uint4*>(w1 + k));
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
      b[i] = there[i] && k < p.K ? *reinterpret_cast<const uint4*>(x[i] + head * p.x.s_h + c) : zero;
    c += 32;
    if (p.x.heads > 1 && c >= p.x.D) c -= p.x.D, ++head;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      mma_16x8<T>(acc[i], a0.x, a1.x, a0.y, a1.y, b[i].x, b[i].y);
      mma_16x8<T>(acc[i], a0.z, a1.z, a0.w, a1.w, b[i].z, b[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    part[warp][i][g][2 * t] = acc[i][0];
    part[warp][i][g][2 * t + 1] = acc[i][1];
    part[warp][i][g + 8][2 * t] = acc[i][2];
    part[warp][i][g + 8][2 * t + 1] = acc[i][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < NT * 8 * kFewColumns; e += 32 * WARPS) {
    const int m = e / kFewColumns, f = e % kFewColumns, col = f0 + f;
    if (m >= M || col >= p.F) continue;
    float v[1] = {0.f};
#pragma unroll
    for (int i = 0; i < WARPS; ++i) v[0] += part[i][m / 8][f][m % 8];
    const int batch = m / p.rows, n = m % p.rows;
    if (p.bias) v[0] += p.bias[col];
    if (p.z.data) *at<T>(p.z, batch, n, col) = static_cast<T>(v[0]);
    activate_n(v, p.act);
    if (p.residual.data) v[0] += static_cast<float>(*at<T>(p.residual, batch, n, col));
    *at<T>(p.out, batch, n, col) = static_cast<T>(v[0]);
  }
}

// ---------------------------------------------------------------- dz and db
// A block takes 256 columns and every blocks_y-th group of 8 rows; a thread 8
// columns, whose sum it keeps.
template <typename T>
__global__ void __launch_bounds__(256) slope_kernel(const SlopeParams p) {
  __shared__ float part[8][32][9];
  ptx::let_next_start();
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int c = (blockIdx.x * 32 + tx) * 8;
  const unsigned M = (unsigned)p.batches * p.rows;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < p.F) {
    const T* const dsrc = at<T>(p.dout, 0, 0, c);
    const T* const zsrc = p.act != kActNone ? at<T>(p.z, 0, 0, c) : nullptr;
    T* const dst = static_cast<T*>(p.dz) + c;
    const unsigned step = gridDim.y * 8;
    const bool act = p.act != kActNone;
    // the rows two ahead are asked for before a row is worked on
    uint4 nd[2], nz[2];
    auto ask = [&](unsigned m, int slot) {
      if (m >= M) return;
      const unsigned b = p.batches > 1 ? p.by_rows(m) : 0, n = m - b * (unsigned)p.rows;
      nd[slot] = *reinterpret_cast<const uint4*>(dsrc + b * p.dout.s_b + n * p.dout.s_n);
      if (act) nz[slot] = *reinterpret_cast<const uint4*>(zsrc + b * p.z.s_b + n * p.z.s_n);
    };
    const unsigned m0 = blockIdx.y * 8 + ty;
    ask(m0, 0);
    ask(m0 + step, 1);
    for (unsigned m = m0; m < M;) {
#pragma unroll
      for (int slot = 0; slot < 2; ++slot, m += step) {
        if (m >= M) break;
        float v[8], z[8];
        unpack8<T>(nd[slot], v);
        if (act) {
          const uint4 q = nz[slot];
          unpack8<T>(make_uint4(finite2<T>(q.x), finite2<T>(q.y), finite2<T>(q.z), finite2<T>(q.w)), z);
        }
        ask(m + 2 * step, slot);
        if (act) {
          times_slope(v, z, p.act);
          *reinterpret_cast<uint4*>(dst + (long long)m * p.F) = pack8<T>(v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
      }
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) part[ty][tx][i] = sum[i];
  __syncthreads();
  const int t = ty * 32 + tx, o = blockIdx.x * 256 + t;
  if (o < p.F) {
    float s = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y) s += part[y][t / 8][t % 8];
    p.partial[(long long)blockIdx.y * p.F + o] = s;
  }
}

// db = sum of the blocks' column sums, 32 columns a block, always in the same order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* partial, int blocks, int F, float* db) {
  ptx::wait_for_previous();
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  if (c < F)
    for (int b = threadIdx.y; b < blocks; b += 32) a += partial[(long long)b * F + c];
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  float v = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int oc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && oc < F) db[oc] = v;
}

template <int KIND, typename T>
cudaError_t launch_gemm(const GemmParams& p, int num_sms, cudaStream_t st) {
  const cudaError_t e = allow_smem<gemm_kernel<KIND, T>>(kGemmSmem);
  if (e != cudaSuccess) return e;
  const long long pairs = p.units < num_sms / 2 ? p.units : num_sms / 2;
  return launch_behind(gemm_kernel<KIND, T>, dim3((unsigned)(2 * pairs)), dim3(kThreads), kGemmSmem, st, p);
}

template <typename T>
cudaError_t launch_gemm_kind(const GemmParams& p, int kind, int num_sms, cudaStream_t st) {
  if (kind == kGemmForward) return launch_gemm<kGemmForward, T>(p, num_sms, st);
  if (kind == kGemmInput) return launch_gemm<kGemmInput, T>(p, num_sms, st);
  return launch_gemm<kGemmWeight, T>(p, num_sms, st);
}

// Sixteen warps a block keep more of W in flight, but fewer blocks fit on an SM
// and more sums are joined. They are taken for rows longer than 2048, and from
// 1024 on where the blocks are few or the rows many (us with eight and sixteen
// warps, W out of memory; one row: 256 -> 4096 3.1 and 3.3, 1024 -> 4096 5.1 and
// 4.4, 1536 -> 1536 5.6 and 4.3, 1536 -> 9216 8.3 and 9.5, 2048 -> 8192 9.6 and
// 11.5, 4096 -> 4096 12.4 and 9.7, 4096 -> 12288 28.8 and 21.5; 16 rows:
// 1536 -> 6144 7.7 and 9.6; 32 rows: 256 -> 9216 7.1 and 8.1, 1536 -> 9216 20.7
// and 14.7).
template <int NT, typename T>
cudaError_t launch_few_tiles(const FewRowsParams& p, cudaStream_t st) {
  const int blocks = (p.F + kFewColumns - 1) / kFewColumns;
  if (p.K > 2048 || (p.K >= 1024 && (NT > 2 || blocks <= 256))) few_rows_kernel<NT, 16, T><<<blocks, 512, 0, st>>>(p);
  else few_rows_kernel<NT, 8, T><<<blocks, 256, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_few(const FewRowsParams& p, cudaStream_t st) {
  const int M = p.batches * p.rows;
  if (M <= 8) return launch_few_tiles<1, T>(p, st);
  if (M <= 16) return launch_few_tiles<2, T>(p, st);
  return launch_few_tiles<4, T>(p, st);
}

}  // namespace

cudaError_t launch_linear_gemm(const GemmParams& p, int kind, int type, int num_sms, cudaStream_t st) {
  return type ? launch_gemm_kind<__half>(p, kind, num_sms, st) : launch_gemm_kind<__nv_bfloat16>(p, kind, num_sms, st);
}

cudaError_t launch_linear_finish(const FinishParams& p, int type, cudaStream_t st) {
  const int grid = p.rest * (p.bn / 8);
  return type ? launch_behind(finish_kernel<__half>, dim3(grid), dim3(256), 0, st, p)
              : launch_behind(finish_kernel<__nv_bfloat16>, dim3(grid), dim3(256), 0, st, p);
}

cudaError_t launch_linear_few_rows(const FewRowsParams& p, int type, cudaStream_t st) {
  return type ? launch_few<__half>(p, st) : launch_few<__nv_bfloat16>(p, st);
}

cudaError_t launch_linear_slope(const SlopeParams& p, int type, float* db, cudaStream_t st) {
  const dim3 grid((p.F + 255) / 256, p.blocks_y), block(32, 8);
  if (type) slope_kernel<__half><<<grid, block, 0, st>>>(p);
  else slope_kernel<__nv_bfloat16><<<grid, block, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial || p.blocks_y == 1) return e;
  return launch_behind(column_sum_kernel, dim3((p.F + 31) / 32), dim3(32, 32), 0, st, (const float*)p.partial,
                       p.blocks_y, p.F, db);
}

cudaError_t linear_failures(unsigned (&counts)[kLinearFailureWords], cudaStream_t st) {
  const cudaError_t e = cudaMemcpyFromSymbolAsync(counts, g_linear_failures, sizeof(counts), 0, cudaMemcpyDeviceToHost, st);
  return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

}  // namespace vsa
