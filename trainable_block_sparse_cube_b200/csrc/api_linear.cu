// Host side of the linear product's entry points of include/vsa.h: argument
// checks, the choice of tiles, tensor maps and launches.
#include <map>
#include <mutex>
#include <utility>

#include "host.cuh"
#include "vsa_common.cuh"

namespace {

using vsa::RowsView;

// vsa_linear_set_limits
thread_local unsigned long long t_wait_ns = 1000000000ull;
thread_local int t_stall = 0;

// Which word counts the failures of a stream's products, and how many of them
// its checks have told of. A product in a graph runs on streams that are not
// known when it is captured: those count in word 0, of which every stream is
// told. Streams beyond the number of words share theirs; each of them is then
// told of all that it counts.
class Failures {
 public:
  // The word for a product about to be enqueued on `st`.
  unsigned word(cudaStream_t st) try {
    Key key;
    if (capturing(st) || !find(st, &key)) return 0;
    std::lock_guard<std::mutex> lock(mutex_);
    return entry(key).word;
  } catch (...) {  // no host memory for the stream's entry
    return 0;
  }

  // Whether products of `st` or of graphs failed since the last look.
  vsa_status look(cudaStream_t st) try {
    Key key;
    if (capturing(st) || !find(st, &key)) return VSA_ERR_CUDA;
    unsigned counts[vsa::kLinearFailureWords];
    if (vsa::linear_failures(counts, st) != cudaSuccess) return VSA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mutex_);
    Entry& e = entry(key);
    Device& d = devices_[key.first];
    const bool own = news(counts[e.word], &e.told, &d.told[e.word]), graphs = news(counts[0], &e.told_graphs, &d.told[0]);
    return own || graphs ? VSA_ERR_TIMEOUT : VSA_OK;
  } catch (...) {
    return VSA_ERR_CUDA;
  }

 private:
  using Key = std::pair<int, unsigned long long>;  // device, the stream's number (never used again)
  struct Entry {
    unsigned word = 0, told = 0, told_graphs = 0;
  };
  struct Device {
    unsigned streams = 0, told[vsa::kLinearFailureWords] = {};  // the highest counts that any stream was told
  };

  static bool capturing(cudaStream_t st) {
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &s) != cudaSuccess) {
      cudaGetLastError();  // the legacy stream beside a capture
      return true;
    }
    return s != cudaStreamCaptureStatusNone;
  }
  static bool find(cudaStream_t st, Key* key) {
    return cudaGetDevice(&key->first) == cudaSuccess && cudaStreamGetId(st, &key->second) == cudaSuccess;
  }
  // A new stream is not told of what others were told before it came.
  Entry& entry(const Key& key) {
    auto [it, fresh] = entries_.try_emplace(key);
    if (fresh) {
      Device& d = devices_[key.first];
      Entry& e = it->second;
      e.word = 1 + d.streams++ % (vsa::kLinearFailureWords - 1);
      e.told = d.told[e.word];
      e.told_graphs = d.told[0];
    }
    return it->second;
  }
  static bool news(unsigned count, unsigned* told, unsigned* told_any) {
    if ((int)(count - *told) <= 0) return false;  // counts may wrap around
    *told = count;
    if ((int)(count - *told_any) > 0) *told_any = count;
    return true;
  }

  std::mutex mutex_;
  std::map<Key, Entry> entries_;
  std::map<int, Device> devices_;
};
Failures& failures() {
  static Failures f;
  return f;
}

inline size_t align_up(size_t x, size_t to = 256) { return (x + to - 1) / to * to; }
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// How a product of `batches` x `rows` x `cols` over `kblocks` 64-long steps is
// cut: `whole` tiles of 256 x bn, and `rest` tiles in `splits` parts each.
struct Tiling {
  int bn, splits;
  long long whole, rest;
};

// The pairs of CTAs run in rounds; costs in cycles, measured at one tile a pair
// (64 steps of 256 x bn, ns a step: bn 64 205, 128 217, 192 395, 256 506, where
// B comes from memory). A step costs the most of
//   its MMA, 2 bn;
//   its loads, 16 KB of A (less with few rows) and bn/16 KB of B, at the 47
//   bytes a cycle that an SM gets of the L2's rate;
//   B's way from memory, at 3400 bytes a cycle for all pairs, those above one
//   another sharing it;
//   400, the issue of a step.
// A round costs its steps, or the epilogue of the tile before, and the start of
// a tile. The last round's tiles are too few for all pairs and are split along
// the contraction, which costs a second kernel that reads the parts (40 x 4096
// x 4096: 64 tiles of 64 columns 17.3 us, 22 of 192 in three parts 13.8). The
// parts may take several rounds where there is more than one column of tiles
// (products with sides drawn from 64 to 7000 and contractions from 10,000 to
// 40,000, where the cost picks that: 29 of them took 0.91 of the time of the
// best cut into one round, 0.70 to 1.09; with one column of tiles 11 took 1.11,
// 1.03 to 1.19).
// `wide` allows only tiles whose second half of columns does not start inside
// a head.
Tiling choose(long long batches, long long rows, long long cols, long long kblocks, int sms, bool wide) {
  const long long pairs = sms / 2, row_tiles = batches * ceil_div(rows, 256);
  const double tile_rows = rows < 256 ? rows : 256;
  Tiling best{};
  double best_cost = -1;
  for (int bn = 256; bn >= 64; bn -= 32) {
    if (wide && bn % 128) continue;
    const long long tiles = row_tiles * ceil_div(cols, bn), whole = tiles / pairs * pairs, rest = tiles - whole;
    const double least[] = {2.0 * bn, (128.0 * (tile_rows < 128 ? tile_rows : 128) + 64.0 * bn) / 47,
                            128.0 * bn * (tiles < pairs ? tiles : pairs) / (row_tiles < 8 ? row_tiles : 8) / 3400};
    double step = 400;
    for (double c : least)
      if (step < c) step = c;
    const double epilogue = 2000 + 25.0 * bn, all = kblocks * step;
    const double base = whole / pairs * ((all > epilogue ? all : epilogue) + 800) + epilogue;
    const long long most = cols <= bn ? pairs : 4 * pairs;  // parts
    for (int s : {1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 24, 32}) {
      if (s > 1 && (s > kblocks || rest * s > most || !rest)) break;
      double cost = base + ceil_div(rest * s, pairs) * (ceil_div(kblocks, s) * step + 800);
      if (s > 1) cost += 2500 + 8.0 * s * rest * tile_rows * bn / 2700;
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best = s > 1 ? Tiling{bn, s, whole, rest} : Tiling{bn, 1, tiles, 0};
      }
    }
  }
  return best;
}

// One product: what a tile needs to know, and the bytes of its parts.
struct Product {
  int kind;
  long long batches, rows, cols, kblocks, kblocks_batch;
  bool wide;
  Tiling t;

  void plan(int sms) { t = choose(batches, rows, cols, kblocks, sms, wide); }
  size_t partial_bytes() const { return (size_t)t.rest * t.splits * 256 * t.bn * 4; }
};

// The batches of a call are one run of rows if every view allows it.
bool joined(int B, int N, std::initializer_list<const vsa_heads*> views) {
  if (B == 1) return true;
  for (const vsa_heads* v : views)
    if (v && v->s_b != (long long)N * v->s_n) return false;
  return true;
}

Product forward_product(const vsa_linear_sizes* s, bool join) {
  Product p{};
  p.kind = vsa::kGemmForward;
  p.batches = join ? 1 : s->B;
  p.rows = join ? (long long)s->B * s->N : s->N;
  p.cols = s->F;
  p.kblocks = ceil_div(s->K, 64);
  return p;
}
Product input_product(const vsa_linear_sizes* s, bool join) {
  Product p = forward_product(s, join);
  p.kind = vsa::kGemmInput;
  p.cols = s->K;
  p.kblocks = ceil_div(s->F, 64);
  return p;
}
Product weight_product(const vsa_linear_sizes* s, bool join, bool wide) {
  Product p{};
  p.kind = vsa::kGemmWeight;
  p.batches = 1;
  p.rows = s->F;
  p.cols = s->K;
  p.kblocks_batch = ceil_div(join ? (long long)s->B * s->N : s->N, 64);
  p.kblocks = p.kblocks_batch * (join ? 1 : s->B);
  p.wide = wide;
  return p;
}

bool few_rows(const vsa_linear_sizes* s) { return (long long)s->B * s->N <= vsa::kFewRows; }

// Blocks along the rows. One for a few rows: it writes db itself and saves a launch.
int slope_blocks(long long M, int F, int sms) {
  if (M <= 64) return 1;
  const long long strips = ceil_div(F, 256), rows = ceil_div(M, 8), most = 8LL * sms / strips;
  return (int)(rows < most ? rows : most > 1 ? most : 1);
}

vsa_status check_sizes(const vsa_linear_sizes* s) {
  if (!s) return VSA_ERR_INVALID_ARG;
  if (s->type != VSA_TYPE_BF16 && s->type != VSA_TYPE_FP16) return VSA_ERR_UNSUPPORTED;
  if (s->B < 0 || s->N < 0 || s->K < 1 || s->F < 1) return VSA_ERR_SHAPE;
  if (s->K % 8 || s->F % 8 || s->K > (1 << 20) || s->F > (1 << 20) || s->B > (1 << 20)) return VSA_ERR_UNSUPPORTED;
  if ((long long)s->B * s->N > (1LL << 30)) return VSA_ERR_UNSUPPORTED;
  return VSA_OK;
}

// A view of B x N rows of `channels`. With several heads a 64-long step must not cross one.
vsa_status check_view(const vsa_heads* v, const vsa_linear_sizes* s, int channels, bool written) {
  if (!v) return VSA_ERR_INVALID_ARG;
  if (v->heads < 1 || channels % v->heads) return VSA_ERR_SHAPE;
  if (v->heads > 1 && channels / v->heads % 64) return VSA_ERR_UNSUPPORTED;
  vsa_status e = vsa::check_heads(v, s->B, s->N, 2, written);
  if (e != VSA_OK) return e;
  for (long long st : {s->B > 1 ? v->s_b : 0, v->heads > 1 ? v->s_h : 0, s->N > 1 ? v->s_n : 0})
    if (st >= (1LL << 38)) return VSA_ERR_UNSUPPORTED;  // the tensor maps' limit is 2^40 bytes
  return VSA_OK;
}

// One token a batch: the batches are the rows. Returns the view to use, a copy in *store if it differs.
const vsa_heads* single_token(const vsa_heads* v, bool swap, vsa_heads* store) {
  if (!v || !swap) return v;
  *store = *v;
  store->s_n = v->s_b;
  store->s_b = 0;
  return store;
}

RowsView rows_view(const vsa_heads* v, int channels) {
  return v ? RowsView{v->data, v->heads, channels / v->heads, v->s_b, v->s_h, v->s_n} : RowsView{};
}
RowsView plain_rows(void* data, long long N, int channels) {
  return RowsView{data, 1, channels, N * channels, channels, channels};
}

// 4-D map (channel of a head, row, head, batch), 128-byte swizzle.
vsa_status encode(CUtensorMap* m, const RowsView& v, long long rows, long long batches, int box_rows, int type) {
  vsa::EncodeTiledFn enc = vsa::get_encode_fn();
  if (!enc) return VSA_ERR_CUDA;
  const cuuint64_t dims[4] = {(cuuint64_t)v.D, (cuuint64_t)rows, (cuuint64_t)v.heads, (cuuint64_t)batches};
  // strides of dimensions of length 1 are not used, but have to be valid
  const cuuint64_t row = (cuuint64_t)v.D * 2;
  const cuuint64_t strides[3] = {rows > 1 ? (cuuint64_t)v.s_n * 2 : row, v.heads > 1 ? (cuuint64_t)v.s_h * 2 : row,
                                 batches > 1 ? (cuuint64_t)v.s_b * 2 : row};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1}, one[4] = {1, 1, 1, 1};
  const CUtensorMapDataType kind = type ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(m, kind, 4, v.data, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? VSA_OK
             : VSA_ERR_CUDA;
}

// Every 16 channels of a row start on a 32-byte boundary. (Strides of
// dimensions of length 1 count too: they only cost the wider access.)
bool aligned32(const RowsView& v) {
  return !v.data || ((reinterpret_cast<uintptr_t>(v.data) & 31u) == 0 && v.D % 16 == 0 &&
                     (v.s_b % 16 | v.s_h % 16 | v.s_n % 16) == 0);
}

struct Epilogue {
  const float* bias;
  int act;
  RowsView residual, z, out;
};

// out = epilogue(A B): A has rows (or, for the weights' gradient, columns of a
// run of rows) of `a`, B those of `b`. `b_rows`: rows of b's map.
vsa_status run_product(const Product& p, int type, const RowsView& a, const RowsView& b, long long b_rows,
                       const Epilogue& ep, void* workspace, int sms, cudaStream_t st) {
  vsa::GemmParams g{};
  const bool weight = p.kind == vsa::kGemmWeight;
  const long long runs = weight ? p.kblocks / p.kblocks_batch : p.batches, run_rows = weight ? b_rows : p.rows;
  const int half = p.t.bn / 2;
  g.a_rows = p.rows < 128 ? (int)ceil_div(p.rows, 8) * 8 : 128;
  vsa_status e = encode(&g.ta, a, run_rows, runs, weight ? 64 : g.a_rows, type);
  // Few rows make a small tile of A: the MMAs then read what lies behind it,
  // other operands inside the ring, for rows that are not stored.
  g.tile_a = weight ? 16384 : g.a_rows * 128;
  g.stage_bytes = g.tile_a + (p.kind == vsa::kGemmForward ? (int)align_up(half * 128, 1024) : (half + 63) / 64 * 8192);
  g.stages = (7 * 32768 - (16384 - g.tile_a)) / g.stage_bytes;
  if (g.stages > vsa::kGemmMaxStages) g.stages = vsa::kGemmMaxStages;
  if (e == VSA_OK) e = encode(&g.tb, b, b_rows, weight ? runs : 1, p.kind == vsa::kGemmForward ? half : 64, type);
  if (e != VSA_OK) return e;
  g.out = ep.out;
  g.residual = ep.residual;
  g.z = ep.z;
  g.partial = static_cast<float*>(workspace);
  g.wide = aligned32(ep.out) && aligned32(ep.residual) && aligned32(ep.z) &&
           (reinterpret_cast<uintptr_t>(workspace) & 31u) == 0;
  g.a_d = a.D;
  g.b_d = b.D;
  g.bn = p.t.bn;
  g.batches = (int)p.batches;
  g.rows = (int)p.rows;
  g.row_tiles = (int)ceil_div(p.rows, 256);
  g.F = (int)p.cols;
  g.kblocks = (int)p.kblocks;
  g.kblocks_batch = (int)p.kblocks_batch;
  g.bias = ep.bias;
  g.act = ep.act;
  g.stall = t_stall;
  g.wait_ns = t_wait_ns;
  g.failures = failures().word(st);
  const long long units = p.t.whole + p.t.rest * p.t.splits, col_tiles = ceil_div(p.cols, p.t.bn);
  if (units >= 1LL << 31) return VSA_ERR_UNSUPPORTED;
  g.order = vsa::TileOrder(g.batches * g.row_tiles, (int)col_tiles);
  g.by_row_tiles = vsa::Divisor(g.row_tiles);
  if (p.t.rest) g.by_rest = vsa::Divisor((uint32_t)p.t.rest);
  g.whole = (int)p.t.whole;
  g.rest = (int)p.t.rest;
  g.splits = p.t.splits;
  g.units = units;
  if (vsa::launch_linear_gemm(g, p.kind, type, sms, st) != cudaSuccess) return VSA_ERR_CUDA;
  if (!p.t.rest) return VSA_OK;
  vsa::FinishParams f{};
  f.partial = static_cast<const float*>(workspace);
  f.first = g.whole;
  f.rest = g.rest;
  f.splits = g.splits;
  f.bn = g.bn;
  f.row_tiles = g.row_tiles;
  f.order = g.order;
  f.rows = g.rows;
  f.F = g.F;
  f.bias = ep.bias;
  f.act = ep.act;
  f.residual = ep.residual;
  f.z = ep.z;
  f.out = ep.out;
  return vsa::launch_linear_finish(f, type, st) == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

vsa_status check_weight(const void* w, long long stride, const vsa_linear_sizes* s) {
  if (!w) return VSA_ERR_INVALID_ARG;
  if (!vsa::aligned16(w)) return VSA_ERR_ALIGN;
  if (s->F > 1 && stride < s->K) return VSA_ERR_INVALID_ARG;
  if (stride % 8) return VSA_ERR_ALIGN;
  if (stride >= (1LL << 38)) return VSA_ERR_UNSUPPORTED;
  return VSA_OK;
}

vsa_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!need) return VSA_OK;
  if (!ws) return VSA_ERR_INVALID_ARG;
  if (!vsa::aligned16(ws)) return VSA_ERR_ALIGN;
  return have < need ? VSA_ERR_INVALID_ARG : VSA_OK;
}

size_t larger(size_t a, size_t b) { return a > b ? a : b; }

// Backward workspace: dz, the blocks' column sums, the parts of a split product.
struct BackwardBytes {
  size_t dz, sums, parts;
  size_t total() const { return dz + sums + parts; }
};
BackwardBytes backward_bytes(const vsa_linear_sizes* s, int act, bool dx, bool dw, bool db, int sms) {
  const long long M = (long long)s->B * s->N;
  BackwardBytes b{};
  if (act != VSA_ACT_NONE) b.dz = align_up((size_t)M * s->F * 2);
  if (db && slope_blocks(M, s->F, sms) > 1) b.sums = align_up((size_t)slope_blocks(M, s->F, sms) * s->F * 4);
  for (bool join : {false, true}) {
    if (dx) {
      Product p = input_product(s, join);
      p.plan(sms);
      b.parts = larger(b.parts, p.partial_bytes());
    }
    for (bool wide : {false, true})
      if (dw) {
        Product p = weight_product(s, join, wide);
        p.plan(sms);
        b.parts = larger(b.parts, p.partial_bytes());
      }
  }
  return b;
}

bool known_activation(int act) { return act >= VSA_ACT_NONE && act <= VSA_ACT_GELU_TANH; }

static_assert(vsa::kActNone == (int)VSA_ACT_NONE && vsa::kActSilu == (int)VSA_ACT_SILU &&
                  vsa::kActGelu == (int)VSA_ACT_GELU && vsa::kActGeluTanh == (int)VSA_ACT_GELU_TANH,
              "ABI activations");

}  // namespace

extern "C" {

size_t vsa_linear_workspace_bytes(const vsa_linear_sizes* sizes) {
  int sms = 0;
  if (check_sizes(sizes) != VSA_OK || vsa::current_device_sms(&sms) != VSA_OK) return 0;
  if (!sizes->B || !sizes->N || few_rows(sizes)) return 0;
  size_t n = 0;
  for (bool join : {false, true}) {
    Product p = forward_product(sizes, join);
    p.plan(sms);
    n = larger(n, p.partial_bytes());
  }
  return n;
}

vsa_status vsa_linear(const vsa_linear_sizes* sizes, const vsa_heads* x, const void* weight, long long weight_stride,
                      const float* bias, int activation, const vsa_heads* residual, const vsa_heads* z,
                      const vsa_heads* out, void* workspace, size_t ws_bytes, void* stream) {
  vsa_status e = check_sizes(sizes);
  if (e != VSA_OK) return e;
  if (!known_activation(activation)) return VSA_ERR_UNSUPPORTED;
  e = check_view(x, sizes, sizes->K, false);
  if (e == VSA_OK) e = check_view(out, sizes, sizes->F, true);
  if (e == VSA_OK && residual)
    e = residual->heads != out->heads ? VSA_ERR_SHAPE : check_view(residual, sizes, sizes->F, false);
  if (e == VSA_OK && z) e = z->heads != out->heads ? VSA_ERR_SHAPE : check_view(z, sizes, sizes->F, true);
  if (e == VSA_OK) e = check_weight(weight, weight_stride, sizes);
  if (e != VSA_OK) return e;
  if (bias && !vsa::aligned16(bias)) return VSA_ERR_ALIGN;
  if (!sizes->B || !sizes->N) return VSA_OK;
  int sms = 0;
  e = vsa::current_device_sms(&sms);
  if (e != VSA_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool swap = sizes->N == 1;
  vsa_linear_sizes rows = *sizes;
  if (swap) rows.N = sizes->B, rows.B = 1;
  sizes = &rows;
  vsa_heads store[4];
  x = single_token(x, swap, store);
  residual = single_token(residual, swap, store + 1);
  z = single_token(z, swap, store + 2);
  out = single_token(out, swap, store + 3);
  Epilogue ep{bias, activation, rows_view(residual, sizes->F), rows_view(z, sizes->F), rows_view(out, sizes->F)};
  const RowsView xv = rows_view(x, sizes->K);
  if (few_rows(sizes)) {
    vsa::FewRowsParams p{};
    p.x = xv;
    p.residual = ep.residual;
    p.z = ep.z;
    p.out = ep.out;
    p.w = weight;
    p.w_stride = weight_stride;
    p.bias = bias;
    p.act = activation;
    p.rows = sizes->N;
    p.batches = sizes->B;
    p.K = sizes->K;
    p.F = sizes->F;
    return vsa::launch_linear_few_rows(p, sizes->type, st) == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
  }
  Product p = forward_product(sizes, joined(sizes->B, sizes->N, {x, residual, z, out}));
  p.plan(sms);
  e = check_workspace(workspace, ws_bytes, p.partial_bytes());
  if (e != VSA_OK) return e;
  const RowsView w{const_cast<void*>(weight), 1, sizes->K, 0, 0, weight_stride};
  return run_product(p, sizes->type, xv, w, sizes->F, ep, workspace, sms, st);
}

size_t vsa_linear_backward_workspace_bytes(const vsa_linear_sizes* sizes, int activation) {
  int sms = 0;
  if (check_sizes(sizes) != VSA_OK || !known_activation(activation)) return 0;
  if (vsa::current_device_sms(&sms) != VSA_OK) return 0;
  if (!sizes->B || !sizes->N) return 0;
  return backward_bytes(sizes, activation, true, true, true, sms).total();
}

vsa_status vsa_linear_backward(const vsa_linear_sizes* sizes, const vsa_heads* x, const void* weight,
                               long long weight_stride, const vsa_heads* z, int activation, const vsa_heads* dout,
                               const vsa_heads* dx, void* dweight, float* dbias, void* workspace, size_t ws_bytes,
                               void* stream) {
  vsa_status e = check_sizes(sizes);
  if (e != VSA_OK) return e;
  if (!known_activation(activation)) return VSA_ERR_UNSUPPORTED;
  e = check_view(dout, sizes, sizes->F, false);
  if (e == VSA_OK && activation != VSA_ACT_NONE)
    e = z && z->heads != dout->heads ? VSA_ERR_SHAPE : check_view(z, sizes, sizes->F, false);
  if (e == VSA_OK && dweight) e = check_view(x, sizes, sizes->K, false);
  if (e == VSA_OK && dx) e = check_view(dx, sizes, sizes->K, true);
  if (e == VSA_OK && dx) e = check_weight(weight, weight_stride, sizes);
  if (e != VSA_OK) return e;
  if ((dweight && !vsa::aligned16(dweight)) || (dbias && !vsa::aligned16(dbias))) return VSA_ERR_ALIGN;
  int sms = 0;
  e = vsa::current_device_sms(&sms);
  if (e != VSA_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int F = sizes->F, K = sizes->K;
  if (!sizes->B || !sizes->N) {  // no rows: the sums are 0
    if (dweight && cudaMemsetAsync(dweight, 0, (size_t)F * K * 2, st) != cudaSuccess) return VSA_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, (size_t)F * 4, st) != cudaSuccess) return VSA_ERR_CUDA;
    return VSA_OK;
  }
  const bool act = activation != VSA_ACT_NONE, swap = sizes->N == 1;
  vsa_linear_sizes rows = *sizes;
  if (swap) rows.N = sizes->B, rows.B = 1;
  sizes = &rows;
  vsa_heads store[4];
  x = single_token(x, swap, store);
  z = single_token(z, swap, store + 1);
  dout = single_token(dout, swap, store + 2);
  dx = single_token(dx, swap, store + 3);
  const BackwardBytes bytes =
      backward_bytes(sizes, activation, dx != nullptr, dweight != nullptr, dbias != nullptr, sms);
  e = check_workspace(workspace, ws_bytes, bytes.total());
  if (e != VSA_OK) return e;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  RowsView dz = rows_view(dout, F);
  vsa_heads dz_heads = *dout;
  if (act || dbias) {
    vsa::SlopeParams s{};
    s.dout = dz;
    if (act) s.z = rows_view(z, F);
    s.dz = ws;
    s.blocks_y = slope_blocks((long long)sizes->B * sizes->N, F, sms);
    s.partial = !dbias ? nullptr : s.blocks_y == 1 ? dbias : reinterpret_cast<float*>(ws + bytes.dz);
    s.act = activation;
    s.batches = sizes->B;
    s.rows = sizes->N;
    s.by_rows = vsa::Divisor(sizes->N);
    s.F = F;
    if (vsa::launch_linear_slope(s, sizes->type, dbias, st) != cudaSuccess) return VSA_ERR_CUDA;
    if (act) {
      dz = plain_rows(ws, sizes->N, F);
      dz_heads = vsa_heads{ws, 1, (long long)sizes->N * F, F, F};
    }
  }
  void* const parts = ws + bytes.dz + bytes.sums;
  const int M = sizes->B * sizes->N;
  if (dx) {
    Product p = input_product(sizes, joined(sizes->B, sizes->N, {&dz_heads, dx}));
    p.plan(sms);
    const RowsView w{const_cast<void*>(weight), 1, K, 0, 0, weight_stride};
    e = run_product(p, sizes->type, dz, w, F, Epilogue{nullptr, 0, {}, {}, rows_view(dx, K)}, parts, sms, st);
    if (e != VSA_OK) return e;
  }
  if (dweight) {
    const bool join = joined(sizes->B, sizes->N, {&dz_heads, x});
    Product p = weight_product(sizes, join, x->heads > 1);
    p.plan(sms);
    e = run_product(p, sizes->type, dz, rows_view(x, K), join ? M : sizes->N,
                    Epilogue{nullptr, 0, {}, {}, plain_rows(dweight, F, K)}, parts, sms, st);
  }
  return e;
}

vsa_status vsa_linear_check(void* stream) {
  int sms = 0;
  const vsa_status e = vsa::current_device_sms(&sms);
  return e == VSA_OK ? failures().look(static_cast<cudaStream_t>(stream)) : e;
}

vsa_status vsa_linear_set_limits(uint64_t wait_ns, int stall) {
  if (!wait_ns || stall < 0 || stall > vsa::kStallLate) return VSA_ERR_INVALID_ARG;
  const uint64_t most = 1000000000000000;  // eleven days: multiples of it fit into 64 bits
  t_wait_ns = wait_ns < most ? wait_ns : most;
  t_stall = stall;
  return VSA_OK;
}

}  // extern "C"
