// Host side of the projection-side entry points of include/vsa.h (rotary
// positions, per-head norm): argument checks and launches. They hold no state.
#include <cmath>
#include <cstring>

#include "host.cuh"
#include "vsa_common.cuh"

namespace {

using vsa::check_heads;

static_assert(vsa::kRopePairs == VSA_ROPE_MAX_PAIRS && vsa::kRopeAxes == VSA_ROPE_MAX_AXES, "ABI limits");

// Radians a position -> turns a position, modulo 2^32, to the nearest 2^-64:
// the frequency's 53 bits times 192 bits of 1 / (2 pi), in whole numbers. Both
// a quotient of doubles and its fraction would be off by 2^-53 of themselves,
// which positions near 2^31 make 2^-22 of a turn, and fast ones more.
vsa::RopePair turns_of(double freq, int axis) {
  static constexpr uint64_t kInverse[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};
  uint64_t f;
  std::memcpy(&f, &freq, 8);
  const int e = (int)(f >> 52 & 0x7ff);  // |freq| = m 2^(e - 1075), e at least 1 there
  const uint64_t m = (f & ((1ull << 52) - 1)) | (uint64_t)(e > 0) << 52;
  uint64_t digits[4], carry = 0;  // of the product, in 2^(e - 1075 - 192)
  for (int i = 0; i < 3; ++i) {
    const unsigned __int128 p = (unsigned __int128)kInverse[i] * m + carry;
    digits[i] = (uint64_t)p;
    carry = (uint64_t)(p >> 64);
  }
  digits[3] = carry;
  const int drop = 192 - 64 + 1075 - (e > 0 ? e : 1);  // 117 at least, as frequencies stay below 2^64
  const auto bits = [&](int i) -> uint64_t {  // 64 of them from the i-th on
    const int w = i / 64, s = i % 64;
    return w > 3 ? 0 : digits[w] >> s | (s && w < 3 ? digits[w + 1] << (64 - s) : 0);
  };
  uint64_t low = bits(drop), high = bits(drop + 64);
  const uint64_t up = bits(drop - 1) & 1;
  low += up, high += up && !low;
  if (freq < 0) low = 0 - low, high = ~high + (low == 0);
  return vsa::RopePair{(uint32_t)low, (uint32_t)(low >> 32), (uint32_t)high, axis};
}

// The parts of RopeParams that every call shares.
vsa_status fill(vsa::RopeParams* p, const vsa_rope_sizes* s, const vsa_rotation* r, const vsa_positions* o) {
  if (!s || !r || !o) return VSA_ERR_INVALID_ARG;
  if (s->type < VSA_TYPE_BF16 || s->type > VSA_TYPE_FP32) return VSA_ERR_UNSUPPORTED;
  if (s->B < 0 || s->N < 0) return VSA_ERR_SHAPE;
  if (s->D < 8 || s->D > 256 || s->D % 8) return VSA_ERR_UNSUPPORTED;
  if (s->B > (1 << 20) || s->N > (1 << 30) || (long long)s->B * s->N > (1LL << 33)) return VSA_ERR_UNSUPPORTED;
  if (r->rot < 0 || r->rot > s->D || r->rot % 2) return VSA_ERR_SHAPE;
  if (!r->interleaved && r->rot % 16) return VSA_ERR_UNSUPPORTED;
  if (r->axes < 1 || r->axes > VSA_ROPE_MAX_AXES) return VSA_ERR_UNSUPPORTED;
  p->wide = 1;
  p->B = s->B;
  p->N = s->N;
  p->D = s->D;
  p->rot = r->rot;
  p->interleaved = r->interleaved != 0;
  p->axes = r->axes;
  for (int j = 0; j < r->rot / 2; ++j) {
    if (r->axis[j] < 0 || r->axis[j] >= r->axes || !(std::fabs(r->freq[j]) < 0x1p64)) return VSA_ERR_INVALID_ARG;
    p->pairs[j] = turns_of(r->freq[j], r->axis[j]);
  }
  if (!o->list) {
    if (r->axes != 3 || o->T < 0 || o->H < 0 || o->W < 0) return VSA_ERR_SHAPE;
    const long long hw = (long long)o->H * o->W;  // each product stays below 2^62: no overflow
    if (!hw || !o->T) return s->N ? VSA_ERR_SHAPE : VSA_OK;
    if (s->N % hw || s->N / hw != o->T) return VSA_ERR_SHAPE;
    p->pos_kind = 0;
    p->H = o->H;
    p->W = o->W;
    p->by_h = vsa::Divisor(o->H);
    p->by_w = vsa::Divisor(o->W);
    for (int a = 0; a < 3; ++a) p->origin[a] = o->origin[a];
  } else {
    if (o->list_type != 0 && o->list_type != 1) return VSA_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(o->list) & 3u) return VSA_ERR_ALIGN;  // read element by element
    if (o->list_batch < 0) return VSA_ERR_INVALID_ARG;
    p->pos_kind = 1 + o->list_type;
    p->pos = o->list;
    p->pos_batch = o->list_batch;
  }
  return VSA_OK;
}

// One of q, k: its input, output and (norm backward) output gradient.
vsa_status add_tensor(vsa::RopeParams* p, int t, int elem, const vsa_heads* in, const vsa_heads* dy,
                      const vsa_heads* out, const float* w) {
  if (!in && !out && !dy) return t ? VSA_OK : VSA_ERR_INVALID_ARG;
  if (!in || !out) return VSA_ERR_INVALID_ARG;
  if (in->heads != out->heads || (dy && dy->heads != in->heads)) return VSA_ERR_SHAPE;
  vsa_status e = check_heads(in, p->B, p->N, elem, false);
  if (e == VSA_OK && dy) e = check_heads(dy, p->B, p->N, elem, false);
  if (e == VSA_OK) e = check_heads(out, p->B, p->N, elem, true);
  if (e != VSA_OK) return e;
  if (w && !vsa::aligned16(w)) return VSA_ERR_ALIGN;
  vsa::RopeTensor& x = p->t[t];
  x.in = in->data;
  x.out = out->data;
  x.w = w;
  x.heads = in->heads;
  x.in_b = in->s_b, x.in_h = in->s_h, x.in_n = in->s_n;
  x.out_b = out->s_b, x.out_h = out->s_h, x.out_n = out->s_n;
  if ((reinterpret_cast<uintptr_t>(out->data) & 31u) || (out->s_b % 8 | out->s_h % 8 | out->s_n % 8)) p->wide = 0;
  if (dy) x.dy = dy->data, x.dy_b = dy->s_b, x.dy_h = dy->s_h, x.dy_n = dy->s_n;
  return VSA_OK;
}

vsa_status run_rope(const vsa_rope_sizes* s, const vsa_rotation* r, const vsa_positions* o, const vsa_heads* q,
                    const vsa_heads* k, const vsa_heads* q_out, const vsa_heads* k_out, bool back, bool norm,
                    const float* wq, const float* wk, float eps, void* stream) {
  vsa::RopeParams p{};
  vsa_status e = fill(&p, s, r, o);
  if (e != VSA_OK) return e;
  if (norm && !(eps >= 0.f && std::isfinite(eps))) return VSA_ERR_INVALID_ARG;
  const int elem = s->type == VSA_TYPE_FP32 ? 4 : 2;
  e = add_tensor(&p, 0, elem, q, nullptr, q_out, wq);
  if (e == VSA_OK) e = add_tensor(&p, 1, elem, k, nullptr, k_out, wk);
  if (e != VSA_OK) return e;
  if (!p.B || !p.N || !(p.t[0].heads + p.t[1].heads)) return VSA_OK;
  int sms = 0;
  e = vsa::current_device_sms(&sms);
  if (e != VSA_OK) return e;
  p.back = back;
  p.norm = norm;
  p.eps = eps;
  return vsa::launch_rope(p, s->type, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VSA_OK : VSA_ERR_CUDA;
}

}  // namespace

extern "C" {

vsa_status vsa_rope(const vsa_rope_sizes* sizes, const vsa_rotation* rotation, const vsa_positions* positions,
                    const vsa_heads* q, const vsa_heads* k, const vsa_heads* q_out, const vsa_heads* k_out,
                    void* stream) {
  return run_rope(sizes, rotation, positions, q, k, q_out, k_out, false, false, nullptr, nullptr, 0.f, stream);
}

vsa_status vsa_rope_backward(const vsa_rope_sizes* sizes, const vsa_rotation* rotation,
                             const vsa_positions* positions, const vsa_heads* dq_out, const vsa_heads* dk_out,
                             const vsa_heads* dq, const vsa_heads* dk, void* stream) {
  return run_rope(sizes, rotation, positions, dq_out, dk_out, dq, dk, true, false, nullptr, nullptr, 0.f, stream);
}

vsa_status vsa_qk_norm_rope(const vsa_rope_sizes* sizes, const vsa_rotation* rotation,
                            const vsa_positions* positions, const vsa_heads* q, const vsa_heads* k,
                            const float* q_weight, const float* k_weight, float eps, const vsa_heads* q_out,
                            const vsa_heads* k_out, void* stream) {
  return run_rope(sizes, rotation, positions, q, k, q_out, k_out, false, true, q_weight, k_weight, eps, stream);
}

size_t vsa_qk_norm_rope_backward_workspace_bytes(int D) {
  int sms = 0;
  if (D < 8 || D > 256 || D % 8 || vsa::current_device_sms(&sms) != VSA_OK) return 0;
  return vsa::norm_rope_partial_bytes(D, sms);
}

vsa_status vsa_qk_norm_rope_backward(const vsa_rope_sizes* sizes, const vsa_rotation* rotation,
                                     const vsa_positions* positions, const vsa_heads* q, const vsa_heads* k,
                                     const float* q_weight, const float* k_weight, float eps,
                                     const vsa_heads* dq_out, const vsa_heads* dk_out, const vsa_heads* dq,
                                     const vsa_heads* dk, float* dq_weight, float* dk_weight, void* workspace,
                                     size_t ws_bytes, void* stream) {
  vsa::RopeParams p{};
  vsa_status e = fill(&p, sizes, rotation, positions);
  if (e != VSA_OK) return e;
  if (!(eps >= 0.f && std::isfinite(eps)) || !dq_out || (k && !dk_out)) return VSA_ERR_INVALID_ARG;
  const int elem = sizes->type == VSA_TYPE_FP32 ? 4 : 2;
  e = add_tensor(&p, 0, elem, q, dq_out, dq, q_weight);
  if (e == VSA_OK) e = add_tensor(&p, 1, elem, k, dk_out, dk, k_weight);
  if (e != VSA_OK) return e;
  if ((dq_weight && !vsa::aligned16(dq_weight)) || (dk_weight && !vsa::aligned16(dk_weight))) return VSA_ERR_ALIGN;
  int sms = 0;
  e = vsa::current_device_sms(&sms);
  if (e != VSA_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!p.B || !p.N || !(p.t[0].heads + p.t[1].heads)) {  // no rows: the sums are 0
    for (float* dw : {dq_weight, dk_weight})
      if (dw && cudaMemsetAsync(dw, 0, (size_t)p.D * 4, st) != cudaSuccess) return VSA_ERR_CUDA;
    return VSA_OK;
  }
  if (!workspace) return VSA_ERR_INVALID_ARG;
  if (!vsa::aligned16(workspace)) return VSA_ERR_ALIGN;
  if (ws_bytes < vsa::norm_rope_partial_bytes(p.D, sms)) return VSA_ERR_INVALID_ARG;
  p.back = 1;
  p.norm = 1;
  p.eps = eps;
  p.partial = static_cast<float*>(workspace);
  return vsa::launch_norm_rope_backward(p, sizes->type, dq_weight, dk_weight, sms, st) == cudaSuccess ? VSA_OK
                                                                                                      : VSA_ERR_CUDA;
}

}  // extern "C"
