// C ABI of the rotary operators (h2o_rotary_*, h2o_rotate_qkv; declared in
// include/h2o.h). Host side only: frequencies, argument checks and launches on the
// current PyTorch stream.
#include <cuda_runtime.h>

#include <cmath>
#include <string>

#include "h2o.h"
#include "host.h"
#include "rotary.h"

static_assert(H2O_ROTARY_MAX_PAIRS == h2o::kRotaryPairs, "pairs of a head");

namespace h2o {
namespace host {
namespace {

constexpr int64_t kMostElements = int64_t{1} << 60;
constexpr double kPi = 3.14159265358979323846;

bool rotated_channels(int dim) { return dim >= 0 && dim % 16 == 0 && dim <= 2 * H2O_ROTARY_MAX_PAIRS; }

// f / (2 pi) without whole turns, in units of 2^-64 of a turn, rounded once; |f| <= 2^53. A long division in
// binary: f = m 2^e is brought down bit by bit, what is left of it by 2 pi kept in units of 2^-120. Those are
// 2^-121 radians off for every whole turn taken, less than 2^-9 of a unit in all at 2^53; what of f lies
// below them is dropped.
constexpr double kMostRadians = 0x1p53;
uint64_t fraction_of_a_turn(double f) {
  using u128 = unsigned __int128;
  constexpr u128 kTwoPi = (static_cast<u128>(0x06487ed5110b4611ull) << 64) | 0xa62633145c06e0e7ull;  // 2 pi 2^120
  constexpr u128 kOne = static_cast<u128>(1) << 120;
  int e;
  const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(std::fabs(f), &e), 53));
  e -= 53;  // |f| = m 2^e
  u128 r = 0;
  for (int x = e + 52; x >= 0; --x) {  // the whole radians, from the top: r = 2 r + bit, by 2 pi
    r = 2 * r + (x >= e && (m >> (x - e) & 1) ? kOne : 0);
    while (r >= kTwoPi) r -= kTwoPi;
  }
  if (e < 0) {  // and what is left below one
    const uint64_t rest = e > -64 ? m & ((uint64_t{1} << -e) - 1) : m;
    r += 120 + e >= 0 ? static_cast<u128>(rest) << (120 + e) : -(120 + e) < 64 ? static_cast<u128>(rest >> -(120 + e)) : 0;
    if (r >= kTwoPi) r -= kTwoPi;
  }
  uint64_t turns = 0;
  for (int i = 0; i < 64; ++i) {
    r *= 2;
    turns = 2 * turns + (r >= kTwoPi);
    if (r >= kTwoPi) r -= kTwoPi;
  }
  turns += 2 * r >= kTwoPi;  // (up to a whole turn, which is none)
  return f < 0 ? 0 - turns : turns;
}

// Bytes from the first to behind the last channel of a view.
size_t extent(const RotateArgs& a, int i) {
  if (!a.heads[i] || !a.n || !a.T) return 0;
  const int64_t last = (a.n - 1) * a.batch[i] + (a.T - 1) * a.token[i] + (a.heads[i] - 1) * a.head[i];
  return (static_cast<size_t>(last) + a.d) * 2;
}

}  // namespace

int rotate_args(const h2o_qkv* x, const h2o_rotary* r, int n, int T, void* const (&out)[3], bool rows, RotateArgs* to) {
  if (!x) return fail(H2O_EINVAL, "null h2o_qkv");
  if (x->head_dim != 64 && x->head_dim != 128) return fail(H2O_EINVAL, "head_dim must be 64 or 128");
  if (T < 0 || T > H2O_MAX_T) return fail(H2O_EINVAL, "T out of range");
  if (static_cast<int64_t>(n) * T >= (int64_t{1} << 31)) return fail(H2O_EINVAL, "2^31 tokens or more");
  RotateArgs& a = *to;
  a.n = n;
  a.T = T;
  a.d = x->head_dim;
  const char* const names[3] = {"q", "k", "v"};
  const h2o_heads* const views[3] = {&x->q, &x->k, &x->v};
  for (int i = 0; i < 3; ++i) {
    const h2o_heads& w = *views[i];
    const int heads = i ? x->heads : x->q_heads;
    const std::string name = names[i];
    if (!w.data) {
      if (out[i]) return fail(H2O_EINVAL, "an output for " + name + ", which is not there");
      continue;
    }
    if (heads < 1 || heads > H2O_ROTARY_MAX_HEADS) return fail(H2O_EINVAL, "heads of " + name + " out of range");
    if ((rows || i == 0) && !out[i]) return fail(H2O_EINVAL, "null output for " + name);
    if (!aligned16(w.data) || !aligned16(out[i])) return fail(H2O_EINVAL, name + " and its output must be 16-byte aligned");
    a.in[i] = w.data;
    a.out[i] = out[i];
    a.heads[i] = heads;
    const int64_t strides[3] = {w.batch, w.token, w.head};
    const int sizes[3] = {n, T, heads};
    int64_t* const mine[3] = {&a.batch[i], &a.token[i], &a.head[i]};
    for (int k = 0; k < 3; ++k) {
      if (sizes[k] > 1 && (strides[k] < 0 || strides[k] % 8 || strides[k] > (int64_t{1} << 30) * x->head_dim))
        return fail(H2O_EINVAL, "strides of " + name + " must be multiples of 8 in [0, 2^30 head_dim]");
      // (the bytes of three dimensions then stay inside 63 bits)
      if (sizes[k] > 1 && strides[k] > kMostElements / (sizes[k] - 1))
        return fail(H2O_EINVAL, "strides of " + name + " reach beyond 2^60 elements");
      *mine[k] = sizes[k] > 1 ? strides[k] : 0;
    }
  }
  a.norm[0] = a.in[0] ? x->q_norm : nullptr;
  a.norm[1] = a.in[1] ? x->k_norm : nullptr;
  if (!aligned16(a.norm[0]) || !aligned16(a.norm[1])) return fail(H2O_EINVAL, "q_norm and k_norm must be 16-byte aligned");
  a.eps = x->eps;
  if ((a.norm[0] || a.norm[1]) && !(a.eps >= 0.f && std::isfinite(a.eps)))
    return fail(H2O_EINVAL, "eps must be finite and not negative");
  a.r.factor = 1.f;
  a.r.half = 1;
  if (r) {
    if (!rotated_channels(r->dim) || r->dim > a.d)
      return fail(H2O_EINVAL, "rotated channels must be a multiple of 16, at most head_dim");
    if (r->layout != H2O_ROTARY_HALF && r->layout != H2O_ROTARY_INTERLEAVED)
      return fail(H2O_EINVAL, "unknown rotary layout");
    if (!std::isfinite(r->factor)) return fail(H2O_EINVAL, "the rotary's factor must be finite");
    a.r.dim = r->dim;
    a.r.half = r->layout == H2O_ROTARY_HALF;
    a.r.factor = r->factor;
    for (int i = 0; i < r->dim / 2; ++i) a.r.turns[i] = r->turns[i];
  }
  // no output may lie on an input or on another output
  for (int i = 0; i < 3; ++i) {
    const size_t bytes = a.out[i] ? static_cast<size_t>(n) * T * a.heads[i] * a.d * 2 : 0;
    for (int j = 0; j < 3; ++j) {
      const size_t other = j < i && a.out[j] ? static_cast<size_t>(n) * T * a.heads[j] * a.d * 2 : 0;
      if (bytes && (overlap(a.out[i], bytes, a.in[j], extent(a, j)) || (other && overlap(a.out[i], bytes, a.out[j], other))))
        return fail(H2O_EINVAL, "outputs must not overlap the inputs or each other");
    }
  }
  return H2O_OK;
}

}  // namespace host
}  // namespace h2o

using namespace h2o::host;

extern "C" {

int h2o_rotary_frequencies(int dim, double base, int scaling, double factor, double original, double low,
                           double high, double* frequencies) {
  if (!frequencies) return fail(H2O_EINVAL, "null frequencies");
  if (!rotated_channels(dim) || dim == 0)
    return fail(H2O_EINVAL, "rotated channels must be a multiple of 16 in [16, 128]");
  if (!(base > 0) || !std::isfinite(base)) return fail(H2O_EINVAL, "base must be positive and finite");
  if (scaling < H2O_ROTARY_PLAIN || scaling > H2O_ROTARY_PARTS) return fail(H2O_EINVAL, "unknown scaling");
  if (scaling != H2O_ROTARY_PLAIN && (!(factor > 0) || !std::isfinite(factor)))
    return fail(H2O_EINVAL, "factor must be positive and finite");
  if (scaling == H2O_ROTARY_PARTS &&
      (!(original > 0) || !std::isfinite(original) || !(high > low) || !std::isfinite(low) || !std::isfinite(high)))
    return fail(H2O_EINVAL, "need original > 0 and high > low");
  if (scaling == H2O_ROTARY_NTK) base *= std::pow(factor, static_cast<double>(dim) / (dim - 2));
  for (int i = 0; i < dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / dim);
    if (scaling == H2O_ROTARY_LINEAR) f /= factor;
    if (scaling == H2O_ROTARY_PARTS) {
      const double share = (original * f / (2 * kPi) - low) / (high - low);
      const double g = share < 0 ? 0 : share > 1 ? 1 : share;
      f = g * f + (1 - g) * f / factor;
    }
    frequencies[i] = f;
  }
  return H2O_OK;
}

int h2o_rotary_init(h2o_rotary* out, int dim, int layout, const double* frequencies, double factor) {
  if (!out) return fail(H2O_EINVAL, "null rotary");
  if (!rotated_channels(dim)) return fail(H2O_EINVAL, "rotated channels must be a multiple of 16 in [0, 128]");
  if (layout != H2O_ROTARY_HALF && layout != H2O_ROTARY_INTERLEAVED) return fail(H2O_EINVAL, "unknown rotary layout");
  if (dim && !frequencies) return fail(H2O_EINVAL, "null frequencies");
  if (!std::isfinite(static_cast<float>(factor))) return fail(H2O_EINVAL, "factor must be finite");
  for (int i = 0; i < dim / 2; ++i)
    if (!(std::fabs(frequencies[i]) <= kMostRadians))
      return fail(H2O_EINVAL, "frequencies must be finite and at most 2^53 radians a position");
  *out = h2o_rotary{};
  out->dim = dim;
  out->layout = layout;
  out->factor = static_cast<float>(factor);
  for (int i = 0; i < dim / 2; ++i) out->turns[i] = fraction_of_a_turn(frequencies[i]);
  return H2O_OK;
}

int h2o_rotate_qkv(const h2o_qkv* x, const h2o_rotary* rotary, int batch, int T, const int32_t* positions,
                   void* q_out, void* k_out, void* v_out) {
  if (batch < 0) return fail(H2O_EINVAL, "batch out of range");
  h2o::RotateArgs a{};
  if (int rc = rotate_args(x, rotary, batch, T, {q_out, k_out, v_out}, true, &a)) return rc;
  a.positions = positions;
  if (batch == 0 || T == 0 || !(a.heads[0] + a.heads[1] + a.heads[2])) return H2O_OK;
  return guarded([&] { return launch_status(h2o::rotate_qkv(a, current_stream()), "rotation launch"); });
}

}  // extern "C"
