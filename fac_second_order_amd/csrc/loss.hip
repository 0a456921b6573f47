// Losses over a model's logits with their gradient in the logits: the clipped policy
// loss with a KL term, and the preference loss over pairs of sequences.
//
// A row of logits z predicts one token y: l = z[y] - log sum_j exp(z_j). Both losses
// are functions of the rows' l, so the gradient of a row is one coefficient times
// (one-hot(y) - softmax(z)). Per element that is two exponentials against four to
// eight bytes moved: HBM-bound.
//
// The softmax is taken about a maximum in fp32. What is formed once per row or per
// sequence (the sum over the waves, l, the ratio, the sums of l) is formed in fp64: l is
// a difference of numbers much larger than the error that a ratio near its bound may carry.
#include "row_ops.hpp"

namespace kfac {

constexpr int LT = 256;    // threads of the blocks that hold no row
constexpr float LOG2E = 1.44269504088896340736f;
// What rounding log2(e) to fp32 leaves off. Without it the exponential of d is off by
// 1.3e-8 d of itself, always to the same side, which a sum of l over a long sequence shows.
constexpr float LOG2E_REST = 1.925963033500e-8f;
constexpr float NEG_INF = -__builtin_huge_valf();

struct LossRows {
  const void* logits;
  void* dlogits;         // NULL: no gradient
  const int64_t* token;
  const uint8_t* mask;   // NULL: every row counts
  const int32_t* begin;  // NULL: one sequence of all rows
  int64_t ld, ld_grad;
  int32_t rows, vocab, seqs;
};

// First and one-past-last row of the sequences [s0, s1), held inside the tensor
// whatever the offsets say.
__device__ inline void seq_range(const LossRows& a, int s0, int s1, int& r0, int& r1) {
  r0 = a.begin ? min(max(gp(a.begin)[s0], 0), a.rows) : 0;
  r1 = a.begin ? min(max(gp(a.begin)[s1], r0), a.rows) : a.rows;
}

// A row counts if its mask is set and its token lies in the vocabulary.
__device__ inline bool row_counts(const LossRows& a, int t) {
  if (a.mask && !gp(a.mask)[t]) return false;
  const int64_t y = gp(a.token)[t];
  return y >= 0 && y < a.vocab;
}

// exp(z - m), the argument off by its rounding alone.
__device__ inline float exp_about(float z, float m) {
  const float d = z - m;
  return __builtin_amdgcn_exp2f(fmaf(d, LOG2E, d * LOG2E_REST));
}

__device__ inline float wave_max(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
template <class V>
__device__ inline V wave_add(V v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <int NT, class V>
__device__ inline V block_add(V v, V* s) {
  v = wave_add(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  V t = 0;
  for (int i = 0; i < NT / 64; ++i) t += s[i];
  return t;
}

// Maximum of a set of logits and the sum of exp(z - maximum).
struct MaxSum {
  float m;
  double s;
};

// The lanes' sets as one, in every lane.
__device__ inline MaxSum join_lanes(MaxSum v) {
  const float m = wave_max(v.m);
  // nothing but -inf: no weight, though a NaN stays in the sum
  const double s = m == NEG_INF ? v.s : v.s * exp(static_cast<double>(v.m) - m);
  return {m, wave_add(s)};
}

// Gradient of a row, coef (one-hot(y) - softmax): -coef softmax(z) everywhere but at y.
template <class T>
struct GradRow {
  typedef typename Chunk16<T>::vec V;
  static constexpr int EV = Chunk16<T>::ev;
  float m, scale;  // 16-bit types: log2(|coef| / sum); fp32: -coef / sum
  float at_y;
  int y;
  unsigned sign;   // flips the signs of two 16-bit results
  __device__ inline GradRow(float m_, double sum, int y_, float z_y, float coef) : m(m_), y(y_) {
    const float inv = static_cast<float>(1.0 / sum);
    at_y = coef * (1.f - exp_about(z_y, m) * inv);
    scale = sizeof(T) == 2 ? __builtin_amdgcn_logf(fabsf(coef) * inv) : -coef * inv;
    sign = coef > 0.f ? 0x80008000u : 0u;
  }
  // fp32 keeps the exponential as exact as the sum's. For 16-bit results the coefficient
  // goes into the exponent, two operations beside the exponential instead of four: that rounds
  // the argument, at most 2^-24 * 150 where the result is not 0, and log2(e), 2^-26 of as much,
  // against half steps of 2^-11 and 2^-8.
  __device__ inline float weight(float z) const {
    return sizeof(T) == 2 ? __builtin_amdgcn_exp2f(fmaf(z - m, LOG2E, scale)) : exp_about(z, m) * scale;
  }
  __device__ inline V group(const V& z, int g) const {
    V w;
#pragma unroll
    for (int u = 0; u < EV; ++u) w[u] = static_cast<T>(weight(static_cast<float>(z[u])));
    if constexpr (sizeof(T) == 2) w = __builtin_bit_cast(V, __builtin_bit_cast(v4u, w) ^ sign);
    if (g == y / EV)
#pragma unroll
      for (int u = 0; u < EV; ++u) w[u] = u == y % EV ? static_cast<T>(at_y) : w[u];
    return w;
  }
  __device__ inline T one(float z, int j) const {
    const float w = weight(z);
    return static_cast<T>(j == y ? at_y : sign && sizeof(T) == 2 ? -w : w);
  }
};

// A row over NT threads, C groups of 16 bytes in each thread's registers: all loads are in
// flight at once and the row is read from memory once. Groups past the row hold -inf, which
// weighs nothing; the last vocab % EV logits, one a thread, are `rest`. A group index that no
// thread reaches is skipped by all. C = 0: the row stays in memory, read twice.
template <class T, int NT, int C>
struct Row {
  typedef typename Chunk16<T>::vec V;
  static constexpr int EV = Chunk16<T>::ev;
  V v[C ? C : 1];
  float rest;

  __device__ inline void load(const KG T* z, int vocab, int tid) {
    const int full = vocab / EV;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * NT < full) {
#pragma unroll
        for (int u = 0; u < EV; ++u) v[c][u] = static_cast<T>(NEG_INF);
        if (c * NT + tid < full) v[c] = *reinterpret_cast<const KG V*>(z + (c * NT + tid) * EV);
      }
    rest = full * EV + tid < vocab ? static_cast<float>(z[full * EV + tid]) : NEG_INF;
  }

  // Of the wave's part of the row, in every lane.
  __device__ inline MaxSum wave_stats(const KG T* z, int vocab, int tid) const {
    const int full = vocab / EV;
    if constexpr (C > 0) {
      float m = rest;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * NT < full)
#pragma unroll
          for (int u = 0; u < EV; ++u) m = fmaxf(m, static_cast<float>(v[c][u]));
      m = wave_max(m);
      const float at = m == NEG_INF ? 0.f : m;
      float s = exp_about(rest, at);
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * NT < full) {
          // opaque, so that the groups are widened again here instead of kept as floats
          v4u raw = __builtin_bit_cast(v4u, v[c]);
          asm("" : "+v"(raw));
          const V x = __builtin_bit_cast(V, raw);
          float e = 0;
#pragma unroll
          for (int u = 0; u < EV; ++u) e += exp_about(static_cast<float>(x[u]), at);
          s += e;
        }
      return {m, wave_add(static_cast<double>(s))};
    } else {  // a running maximum in each thread, the sum about it in fp64
      float m = rest;
      double s = rest == NEG_INF ? 0.0 : exp_about(rest, rest);
      for (int g = tid; g < full; g += NT) {
        const V x = *reinterpret_cast<const KG V*>(z + int64_t(g) * EV);
        float top = m;
#pragma unroll
        for (int u = 0; u < EV; ++u) top = fmaxf(top, static_cast<float>(x[u]));
        const float at = top == NEG_INF ? 0.f : top;
        if (top != m) s *= exp(static_cast<double>(m) - at);
        m = top;
        float e = 0;
#pragma unroll
        for (int u = 0; u < EV; ++u) e += exp_about(static_cast<float>(x[u]), at);
        s += e;
      }
      return join_lanes({m, s});
    }
  }

  // An element is read and written by one thread: d may be z.
  __device__ inline void gradient(const GradRow<T>& k, const KG T* z, KG T* d, int vocab, int tid) const {
    const int full = vocab / EV;
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * NT + tid < full) {
          const int g = c * NT + tid;
          *reinterpret_cast<KG V*>(d + g * EV) = k.group(v[c], g);
        }
    } else {
      for (int g = tid; g < full; g += NT) {
        const V x = *reinterpret_cast<const KG V*>(z + int64_t(g) * EV);
        *reinterpret_cast<KG V*>(d + int64_t(g) * EV) = k.group(x, g);
      }
    }
    if (full * EV + tid < vocab) d[full * EV + tid] = k.one(rest, full * EV + tid);
  }
};

template <class T, int NT>
__device__ inline void row_zero(KG T* d, int vocab, int tid) {
  typedef typename Chunk16<T>::vec V;
  constexpr int EV = Chunk16<T>::ev;
  const int full = vocab / EV;
  const V w = {};
  for (int g = tid; g < full; g += NT) *reinterpret_cast<KG V*>(d + int64_t(g) * EV) = w;
  if (full * EV + tid < vocab) d[full * EV + tid] = static_cast<T>(0.f);
}

// A row's block: a wave for a short row (four rows a block, no barrier), else a block.
template <int NT>
constexpr int kRowsPerBlock = NT == 64 ? 4 : 1;
template <int NT>
constexpr int kRowThreads = NT == 64 ? 256 : NT;

// The waves' statistics as the row's, in the row's first wave.
template <int NT>
__device__ inline MaxSum join_waves(MaxSum v, MaxSum* lds) {
  if constexpr (NT > 64) {
    const int lane = threadIdx.x & 63;
    if (lane == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x < 64) {
      v = lane < NT / 64 ? lds[lane] : MaxSum{NEG_INF, 0.0};
      v = join_lanes(v);
    }
  }
  return v;
}

// Sequence q in `slices` parts: how many rows of each count; per row: its sequence, -1
// where it does not count and -2 outside every sequence.
__global__ void __launch_bounds__(LT) loss_count_kernel(LossRows a, int32_t* __restrict__ row_seq,
                                                        int32_t* __restrict__ count) {
  __shared__ int s[LT / 64];
  const int q = blockIdx.x, slice = blockIdx.y, slices = gridDim.y;
  int r0, r1, n = 0;
  seq_range(a, q, q + 1, r0, r1);
  const int per = (r1 - r0 + slices - 1) / slices;
  const int b0 = min(r0 + slice * per, r1), b1 = min(b0 + per, r1);
  for (int t = b0 + threadIdx.x; t < b1; t += LT) {
    const bool counts = row_counts(a, t);
    row_seq[t] = counts ? q : -1;
    n += counts;
  }
  n = block_add<LT>(n, s);
  if (threadIdx.x == 0) count[q * slices + slice] = n;
  if (q == 0 && slice == 0)
    for (int t = threadIdx.x; t < r0; t += LT) row_seq[t] = -2;
  if (q == a.seqs - 1 && slice == 0)
    for (int t = r1 + threadIdx.x; t < a.rows; t += LT) row_seq[t] = -2;
}

struct PolicyArgs {
  const float* old_logp;
  const float* ref_logp;  // NULL: no KL term
  const float* advantage;
  float* logp;
  float low, high, kl_coef, grad_scale;
  int32_t by_seq;
};

struct PolicyTerms {
  double part, kl, over;  // weighted surrogate loss, KL and clipped share of a row
};

// Rows that count: all of them, or with by_seq the sequences that have one; a wave's work.
__device__ inline int counted_total(const int32_t* count, int seqs, int slices, bool by_seq) {
  int n = 0;
  for (int i = threadIdx.x & 63; i < (by_seq ? seqs : seqs * slices); i += 64) {
    if (by_seq) {
      int k = 0;
      for (int j = 0; j < slices; ++j) k |= count[i * slices + j];
      n += k != 0;
    } else {
      n += count[i];
    }
  }
  return wave_add(n);
}

template <class T, int NT, int C>
__global__ void __launch_bounds__(kRowThreads<NT>) policy_rows_kernel(LossRows a, PolicyArgs p,
                                                                      const int32_t* __restrict__ row_seq,
                                                                      const int32_t* __restrict__ count, int slices,
                                                                      PolicyTerms* __restrict__ terms) {
  __shared__ MaxSum lds[NT / 64];
  __shared__ struct { double s; float m, coef; } row_s;
  const int tid = threadIdx.x & (NT - 1);
  const int t = blockIdx.x * kRowsPerBlock<NT> + (NT == 64 ? threadIdx.x >> 6 : 0);
  if (t >= a.rows) return;
  int q = row_seq[t];
  if (q >= 0 && (q >= a.seqs || !row_counts(a, t))) q = -2;  // offsets that decrease: no sequence wrote this row
  KG T* d = a.dlogits ? gp(static_cast<T*>(a.dlogits)) + t * a.ld_grad : nullptr;
  if (q < 0) {  // outside (left as it is) or not counted (no gradient)
    if (tid == 0) {
      terms[t] = {0, 0, 0};
      if (q == -1) gp(p.logp)[t] = 0.f;
    }
    if (q == -1 && d) row_zero<T, NT>(d, a.vocab, tid);
    return;
  }
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  const int y = static_cast<int>(gp(a.token)[t]);
  const float z_y = static_cast<float>(z[y]);
  Row<T, NT, C> row;
  row.load(z, a.vocab, tid);
  MaxSum r = join_waves<NT>(row.wave_stats(z, a.vocab, tid), lds);
  float coef = 0;
  if (tid < 64) {
    const int n = counted_total(count, a.seqs, slices, p.by_seq);
    int own = 0;
    for (int j = 0; j < slices; ++j) own += count[q * slices + j];
    const double weight = p.by_seq ? 1.0 / (static_cast<double>(n) * own) : 1.0 / n;
    const double l = static_cast<double>(z_y) - r.m - log(r.s);
    const double ratio = exp(l - gp(p.old_logp)[t]);
    const double adv = gp(p.advantage)[t];
    // NaN goes through: a comparison with it is false
    const double bounded = ratio < 1.0 - p.low ? 1.0 - p.low : ratio > 1.0 + p.high ? 1.0 + p.high : ratio;
    const double free = ratio * adv, held = bounded * adv;
    const bool over = free > held;
    double slope = over ? 0.0 : -free, kl = 0;
    if (p.ref_logp) {
      const double x = gp(p.ref_logp)[t] - l, e = expm1(x);
      kl = e - x;
      if (p.kl_coef != 0.f) slope -= p.kl_coef * e;
    }
    coef = static_cast<float>(p.grad_scale * weight * slope);
    if (tid == 0) {
      gp(p.logp)[t] = static_cast<float>(l);
      terms[t] = {weight * -(over ? held : free), weight * kl, over ? weight : 0.0};
      row_s.s = r.s;
      row_s.m = r.m;
      row_s.coef = coef;
    }
  }
  if (!d) return;
  if constexpr (NT > 64) {
    __syncthreads();
    r.m = row_s.m;
    r.s = row_s.s;
    coef = row_s.coef;
  }
  row.gradient(GradRow<T>(r.m, r.s, y, z_y, coef), z, d, a.vocab, tid);
}

// stats: loss, its surrogate part, the mean KL, the clipped share.
constexpr int FT = 1024;
__global__ void __launch_bounds__(FT) policy_finish_kernel(const PolicyTerms* __restrict__ terms, int rows,
                                                           float kl_coef, float* stats) {
  __shared__ double s[FT / 64];
  double part = 0, kl = 0, over = 0;
  for (int t = threadIdx.x; t < rows; t += FT) {
    part += terms[t].part;
    kl += terms[t].kl;
    over += terms[t].over;
  }
  part = block_add<FT>(part, s);
  kl = block_add<FT>(kl, s);
  over = block_add<FT>(over, s);
  if (threadIdx.x == 0) {
    stats[0] = static_cast<float>(kl_coef != 0.f ? part + kl_coef * kl : part);
    stats[1] = static_cast<float>(part);
    stats[2] = static_cast<float>(kl);
    stats[3] = static_cast<float>(over);
  }
}

// What the gradient of a row needs of its softmax.
struct RowStat {
  float m, z_y;
  double s;
};

// Softmax maximum and sum, and l, of every row that counts and lies in a sequence.
template <class T, int NT, int C>
__global__ void __launch_bounds__(kRowThreads<NT>) pref_rows_kernel(LossRows a, RowStat* __restrict__ row_stat,
                                                                    double* __restrict__ row_logp) {
  __shared__ MaxSum lds[NT / 64];
  const int tid = threadIdx.x & (NT - 1);
  const int t = blockIdx.x * kRowsPerBlock<NT> + (NT == 64 ? threadIdx.x >> 6 : 0);
  if (t >= a.rows) return;
  int r0, r1;
  seq_range(a, 0, a.seqs, r0, r1);
  if (t < r0 || t >= r1) return;
  if (!row_counts(a, t)) {
    if (tid == 0) row_logp[t] = 0;
    return;
  }
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  const float z_y = static_cast<float>(z[gp(a.token)[t]]);
  Row<T, NT, C> row;
  row.load(z, a.vocab, tid);
  const MaxSum r = join_waves<NT>(row.wave_stats(z, a.vocab, tid), lds);
  if (tid == 0) {
    row_stat[t] = {r.m, z_y, r.s};
    row_logp[t] = static_cast<double>(z_y) - r.m - log(r.s);
  }
}

struct PrefArgs {
  const float* ref_logp;  // NULL: zeros
  float* seq_logp;
  float* margin;
  float* loss;
  float beta, smooth, grad_scale;
  int32_t pairs;
};

// log(1 + exp(x))
__device__ inline double softplus(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }

// A block takes PAIRS pairs, a wave each of their sequences: the sums of l, the margins, the
// loss, and for each row the coefficient of its gradient. part: a block's share of the loss.
constexpr int PAIRS = 8;
constexpr int PT = 2 * PAIRS * 64;
__global__ void __launch_bounds__(PT) pref_pairs_kernel(LossRows a, PrefArgs p, const double* __restrict__ row_logp,
                                                        float* __restrict__ row_coef, double* __restrict__ part) {
  __shared__ double sum_s[2 * PAIRS], loss_s[PAIRS];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int local = wave >> 1, side = wave & 1;  // side 1: the other of the pair
  const int i = blockIdx.x * PAIRS + local;
  const bool here = i < p.pairs;
  int r0 = 0, r1 = 0;
  if (here) seq_range(a, i + side * p.pairs, i + side * p.pairs + 1, r0, r1);
  double v = 0;
  for (int t = r0 + lane; t < r1; t += 64) v += row_logp[t];
  v = wave_add(v);
  if (lane == 0) sum_s[wave] = v;
  __syncthreads();
  double loss = 0;
  if (here) {
    const double chosen = sum_s[2 * local], other = sum_s[2 * local + 1];
    const double rc = p.ref_logp ? gp(p.ref_logp)[i] : 0.f, rr = p.ref_logp ? gp(p.ref_logp)[i + p.pairs] : 0.f;
    const double x = p.beta * ((chosen - rc) - (other - rr)), e = p.smooth;
    const double below = softplus(-x), above = softplus(x);  // -log sig(x), -log sig(-x)
    loss = (e != 0 ? (1 - e) * below + e * above : below) / p.pairs;
    const double slope = (e - exp(-above)) * p.beta / p.pairs;
    if (lane == 0) {
      if (side == 0) gp(p.margin)[i] = static_cast<float>(x);
      gp(p.seq_logp)[i + side * p.pairs] = static_cast<float>(v);
    }
    const float c = static_cast<float>(p.grad_scale * (side ? -slope : slope));
    for (int t = r0 + lane; t < r1; t += 64) row_coef[t] = c;
  }
  if (lane == 0 && side == 0) loss_s[local] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0;
    for (int k = 0; k < PAIRS; ++k) total += loss_s[k];
    if (gridDim.x == 1) gp(p.loss)[0] = static_cast<float>(total);
    else part[blockIdx.x] = total;
  }
}

__global__ void __launch_bounds__(LT) pref_finish_kernel(const double* __restrict__ part, int n, float* loss) {
  __shared__ double s[LT / 64];
  double v = 0;
  for (int i = threadIdx.x; i < n; i += LT) v += part[i];
  v = block_add<LT>(v, s);
  if (threadIdx.x == 0) loss[0] = static_cast<float>(v);
}

// Elementwise over the rows, last rows first: what pref_rows_kernel read last is what the
// caches still hold. A block takes LT * GRAD_U groups of 16 bytes of a row.
constexpr int GRAD_U = 2;
template <class T>
__global__ void __launch_bounds__(LT) pref_grad_kernel(LossRows a, const RowStat* __restrict__ row_stat,
                                                       const float* __restrict__ row_coef) {
  typedef typename Chunk16<T>::vec V;
  constexpr int EV = Chunk16<T>::ev;
  int r0, r1;
  seq_range(a, 0, a.seqs, r0, r1);
  const int full = a.vocab / EV, g0 = blockIdx.x * LT * GRAD_U + threadIdx.x;
  const bool last = blockIdx.x == 0 && full * EV + static_cast<int>(threadIdx.x) < a.vocab;
  for (int t = r1 - 1 - static_cast<int>(blockIdx.y); t >= r0; t -= gridDim.y) {
    const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
    KG T* d = gp(static_cast<T*>(a.dlogits)) + t * a.ld_grad;
    if (!row_counts(a, t)) {
      const V none = {};
#pragma unroll
      for (int u = 0; u < GRAD_U; ++u)
        if (g0 + u * LT < full) *reinterpret_cast<KG V*>(d + int64_t(g0 + u * LT) * EV) = none;
      if (last) d[full * EV + threadIdx.x] = static_cast<T>(0.f);
      continue;
    }
    const RowStat r = row_stat[t];
    V v[GRAD_U];
#pragma unroll
    for (int u = 0; u < GRAD_U; ++u)
      if (g0 + u * LT < full) v[u] = *reinterpret_cast<const KG V*>(z + int64_t(g0 + u * LT) * EV);
    const GradRow<T> k(r.m, r.s, static_cast<int>(gp(a.token)[t]), r.z_y, row_coef[t]);
#pragma unroll
    for (int u = 0; u < GRAD_U; ++u)
      if (g0 + u * LT < full) *reinterpret_cast<KG V*>(d + int64_t(g0 + u * LT) * EV) = k.group(v[u], g0 + u * LT);
    if (last) {
      const int j = full * EV + threadIdx.x;
      d[j] = k.one(static_cast<float>(z[j]), j);
    }
  }
}

}  // namespace kfac

using namespace kfac;

static kfac_status rows_validate(int32_t rows, int32_t vocab, int32_t seqs) {
  if (rows < 0) return fail(KFAC_ERR_INVALID, "rows must be >= 0");
  if (vocab < 1 || vocab > (1 << 30)) return fail(KFAC_ERR_INVALID, "vocab = %d out of range", vocab);
  if (seqs < 0 || seqs > (1 << 24)) return fail(KFAC_ERR_INVALID, "%d sequences: out of range", seqs);
  return KFAC_OK;
}

static kfac_status check_array(const void* p, int size, const char* what) {
  if (!p) return fail(KFAC_ERR_INVALID, "%s is NULL", what);
  if (reinterpret_cast<uintptr_t>(p) % size) return fail(KFAC_ERR_INVALID, "%s is misaligned", what);
  return KFAC_OK;
}

// Types, pitches and pointers of the rows of either loss.
static kfac_status rows_check(const LossRows& a, kfac_dtype dtype) {
  if (dtype != KFAC_F16 && dtype != KFAC_F32 && dtype != KFAC_BF16)
    return fail(KFAC_ERR_UNSUPPORTED, "dtype %d is not supported", dtype);
  if (a.rows == 0) return KFAC_OK;
  const int size = dtype == KFAC_F32 ? 4 : 2;
  kfac_status st;
  if ((st = check_array(a.logits, size, "logits")) || (st = check_array(a.token, 8, "token"))) return st;
  if (a.dlogits && (st = check_array(a.dlogits, size, "dlogits"))) return st;
  if (a.begin && (st = check_array(a.begin, 4, "seq_begin"))) return st;
  const int64_t most = int64_t(1) << 40;
  if (a.ld < a.vocab || a.ld > most || (a.dlogits && (a.ld_grad < a.vocab || a.ld_grad > most)))
    return fail(KFAC_ERR_INVALID, "a row pitch is smaller than vocab or out of range");
  if (a.dlogits) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.logits), y = reinterpret_cast<uintptr_t>(a.dlogits);
    const uintptr_t nx = (uintptr_t(a.rows - 1) * a.ld + a.vocab) * size;
    const uintptr_t ny = (uintptr_t(a.rows - 1) * a.ld_grad + a.vocab) * size;
    if (x < y + ny && y < x + nx && !(x == y && a.ld == a.ld_grad))
      return fail(KFAC_ERR_INVALID, "dlogits overlaps logits without being it");
  }
  return KFAC_OK;
}

static bool finite(float x) { return x - x == 0.f; }

// LAUNCH(type) for the type of a code.
#define KFAC_BY_TYPE(dtype, LAUNCH)              \
  do {                                           \
    if ((dtype) == KFAC_F32) { LAUNCH(float) }   \
    else if ((dtype) == KFAC_BF16) { LAUNCH(__bf16) } \
    else { LAUNCH(_Float16) }                    \
  } while (0)

// LAUNCH(T, NT, C) for a row length: as few threads as hold the row in at most 8 groups of
// 16 bytes each (32 registers, eight waves of a SIMD's 16 stay resident), at most 1024; 20
// groups a thread are the most that leave no spills under the 128 registers of a 1024-thread
// block. Longer rows stay in memory.
#define KFAC_BY_ROW(T, vocab, LAUNCH)                     \
  do {                                                    \
    const int groups_ = (vocab) / Chunk16<T>::ev;         \
    if (groups_ <= 64 * 4) { LAUNCH(T, 64, 4) }           \
    else if (groups_ <= 256 * 4) { LAUNCH(T, 256, 4) }    \
    else if (groups_ <= 256 * 8) { LAUNCH(T, 256, 8) }    \
    else if (groups_ <= 512 * 8) { LAUNCH(T, 512, 8) }    \
    else if (groups_ <= 1024 * 8) { LAUNCH(T, 1024, 8) }  \
    else if (groups_ <= 1024 * 16) { LAUNCH(T, 1024, 16) } \
    else if (groups_ <= 1024 * 20) { LAUNCH(T, 1024, 20) } \
    else { LAUNCH(T, 1024, 0) }                           \
  } while (0)

// Parts of a sequence that are counted side by side.
static int count_slices(int32_t rows, int32_t seqs) {
  const int64_t n = rows / (int64_t(seqs) * 1024);
  return n < 1 ? 1 : n > 16 ? 16 : static_cast<int>(n);
}

struct PolicyWs {
  int32_t *row_seq, *count;
  PolicyTerms* terms;
  size_t bytes;
};
static PolicyWs policy_ws(void* ws, int32_t rows, int32_t seqs) {
  Carver cv(ws);
  PolicyWs w;
  w.row_seq = cv.take<int32_t>(rows);
  w.count = cv.take<int32_t>(size_t(seqs ? seqs : 1) * count_slices(rows, seqs ? seqs : 1));
  w.terms = cv.take<PolicyTerms>(rows);
  w.bytes = cv.used;
  return w;
}

extern "C" kfac_status kfac_policy_loss_workspace(int32_t rows, int32_t vocab, int32_t seqs, size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  kfac_status st = rows_validate(rows, vocab, seqs);
  if (st) return st;
  *bytes = policy_ws(nullptr, rows, seqs).bytes;
  return KFAC_OK;
}

extern "C" kfac_status kfac_policy_loss(int32_t rows, int32_t vocab, kfac_dtype dtype, const void* logits, int64_t ld,
                                        const int64_t* token, const uint8_t* mask, int32_t seqs,
                                        const int32_t* seq_begin, const float* old_logp, const float* ref_logp,
                                        const float* advantage, float clip_low, float clip_high, float kl_coef,
                                        int32_t by_sequence, float grad_scale, float* logp, float* stats,
                                        void* dlogits, int64_t ld_grad, void* workspace, size_t ws_bytes,
                                        void* stream) {
  kfac_status st = rows_validate(rows, vocab, seqs);
  if (st) return st;
  if (!(clip_low >= 0.f && clip_low <= 1.f && clip_high >= 0.f && finite(clip_high)))
    return fail(KFAC_ERR_INVALID, "clip_low must be in [0, 1] and clip_high finite and >= 0");
  if (!finite(kl_coef) || !finite(grad_scale)) return fail(KFAC_ERR_INVALID, "kl_coef and grad_scale must be finite");
  if (kl_coef != 0.f && !ref_logp) return fail(KFAC_ERR_INVALID, "a KL term needs ref_logp");
  if (by_sequence != 0 && by_sequence != 1) return fail(KFAC_ERR_INVALID, "by_sequence must be 0 or 1");
  if ((seqs == 0) != (seq_begin == nullptr)) return fail(KFAC_ERR_INVALID, "seqs and seq_begin go together");
  LossRows a = {logits, dlogits, token, mask, seq_begin, ld, ld_grad, rows, vocab, seqs ? seqs : 1};
  if ((st = rows_check(a, dtype)) || (st = check_array(stats, 4, "stats"))) return st;
  if (rows > 0) {
    if ((st = check_array(old_logp, 4, "old_logp")) || (st = check_array(advantage, 4, "advantage")) ||
        (st = check_array(logp, 4, "logp")))
      return st;
    if (ref_logp && (st = check_array(ref_logp, 4, "ref_logp"))) return st;
  }
  if ((st = check_device())) return st;
  const PolicyWs w = policy_ws(workspace, rows, seqs);
  if ((st = check_workspace(workspace, ws_bytes, w.bytes))) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows > 0) {
    const PolicyArgs p = {old_logp, ref_logp, advantage, logp, clip_low, clip_high, kl_coef, grad_scale, by_sequence};
    const int slices = count_slices(rows, a.seqs);
    KFAC_LAUNCH(K_LOSS_COUNT, loss_count_kernel, dim3(a.seqs, slices), dim3(LT), 0, s, a, w.row_seq, w.count);
    KFAC_CHECK_LAUNCH("loss_count_kernel");
#define KFAC_ROWS(T, NT, C)                                                                                      \
  KFAC_LAUNCH(K_POLICY_ROWS, (policy_rows_kernel<T, NT, C>), dim3((rows - 1) / kRowsPerBlock<NT> + 1),           \
              dim3(kRowThreads<NT>), 0, s, a, p, w.row_seq, w.count, slices, w.terms);
#define KFAC_TYPED(T) KFAC_BY_ROW(T, vocab, KFAC_ROWS);
    KFAC_BY_TYPE(dtype, KFAC_TYPED);
#undef KFAC_TYPED
#undef KFAC_ROWS
    KFAC_CHECK_LAUNCH("policy_rows_kernel");
  }
  KFAC_LAUNCH(K_POLICY_FINISH, policy_finish_kernel, dim3(1), dim3(FT), 0, s, w.terms, rows, kl_coef, stats);
  KFAC_CHECK_LAUNCH("policy_finish_kernel");
  return KFAC_OK;
}

struct PrefWs {
  RowStat* stat;
  double *logp, *part;
  float* coef;
  size_t bytes;
};
static int pair_blocks(int32_t pairs) { return pairs < 1 ? 1 : (pairs - 1) / PAIRS + 1; }

static PrefWs pref_ws(void* ws, int32_t rows, int32_t pairs) {
  Carver cv(ws);
  PrefWs w;
  w.stat = cv.take<RowStat>(rows);
  w.logp = cv.take<double>(rows);
  w.part = cv.take<double>(pair_blocks(pairs));
  w.coef = cv.take<float>(rows);
  w.bytes = cv.used;
  return w;
}

extern "C" kfac_status kfac_preference_loss_workspace(int32_t rows, int32_t vocab, int32_t pairs, size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  if (pairs < 0 || pairs > (1 << 23)) return fail(KFAC_ERR_INVALID, "%d pairs: out of range", pairs);
  kfac_status st = rows_validate(rows, vocab, 2 * pairs);
  if (st) return st;
  *bytes = pref_ws(nullptr, rows, pairs).bytes;
  return KFAC_OK;
}

extern "C" kfac_status kfac_preference_loss(int32_t rows, int32_t vocab, kfac_dtype dtype, const void* logits,
                                            int64_t ld, const int64_t* token, const uint8_t* mask, int32_t pairs,
                                            const int32_t* seq_begin, const float* ref_logp, float beta,
                                            float label_smoothing, float grad_scale, float* seq_logp, float* margin,
                                            float* loss, void* dlogits, int64_t ld_grad, void* workspace,
                                            size_t ws_bytes, void* stream) {
  if (pairs < 0 || pairs > (1 << 23)) return fail(KFAC_ERR_INVALID, "%d pairs: out of range", pairs);
  kfac_status st = rows_validate(rows, vocab, 2 * pairs);
  if (st) return st;
  if (!finite(beta) || !finite(grad_scale)) return fail(KFAC_ERR_INVALID, "beta and grad_scale must be finite");
  if (!(label_smoothing >= 0.f && label_smoothing <= 1.f))
    return fail(KFAC_ERR_INVALID, "label_smoothing must be in [0, 1]");
  LossRows a = {logits, dlogits, token, mask, seq_begin, ld, ld_grad, rows, vocab, 2 * pairs};
  if ((st = rows_check(a, dtype)) || (st = check_array(loss, 4, "loss"))) return st;
  if (pairs > 0) {
    if ((st = check_array(seq_begin, 4, "seq_begin")) || (st = check_array(seq_logp, 4, "seq_logp")) ||
        (st = check_array(margin, 4, "margin")))
      return st;
    if (ref_logp && (st = check_array(ref_logp, 4, "ref_logp"))) return st;
  }
  if ((st = check_device())) return st;
  const PrefWs w = pref_ws(workspace, rows, pairs);
  if ((st = check_workspace(workspace, ws_bytes, w.bytes))) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const PrefArgs p = {ref_logp, seq_logp, margin, loss, beta, label_smoothing, grad_scale, pairs};
  const bool any = rows > 0 && pairs > 0;
  if (any) {
#define KFAC_ROWS(T, NT, C)                                                                                 \
  KFAC_LAUNCH(K_PREF_ROWS, (pref_rows_kernel<T, NT, C>), dim3((rows - 1) / kRowsPerBlock<NT> + 1),          \
              dim3(kRowThreads<NT>), 0, s, a, w.stat, w.logp);
#define KFAC_TYPED(T) KFAC_BY_ROW(T, vocab, KFAC_ROWS);
    KFAC_BY_TYPE(dtype, KFAC_TYPED);
#undef KFAC_TYPED
#undef KFAC_ROWS
    KFAC_CHECK_LAUNCH("pref_rows_kernel");
  }
  const int blocks = pair_blocks(pairs);
  KFAC_LAUNCH(K_PREF_PAIRS, pref_pairs_kernel, dim3(blocks), dim3(PT), 0, s, a, p, w.logp, w.coef, w.part);
  KFAC_CHECK_LAUNCH("pref_pairs_kernel");
  if (blocks > 1) {
    KFAC_LAUNCH(K_PREF_FINISH, pref_finish_kernel, dim3(1), dim3(LT), 0, s, w.part, blocks, loss);
    KFAC_CHECK_LAUNCH("pref_finish_kernel");
  }
  if (any && dlogits) {
    const unsigned y = rows < 65535 ? rows : 65535;
#define KFAC_TYPED(T)                                                                                             \
  KFAC_LAUNCH(K_PREF_GRAD, pref_grad_kernel<T>, dim3((vocab / Chunk16<T>::ev) / (LT * GRAD_U) + 1, y), dim3(LT), 0, s, \
              a, w.stat, w.coef);
    KFAC_BY_TYPE(dtype, KFAC_TYPED);
#undef KFAC_TYPED
    KFAC_CHECK_LAUNCH("pref_grad_kernel");
  }
  return KFAC_OK;
}
