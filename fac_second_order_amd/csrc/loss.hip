// Losses over a model's logits with their gradient in the logits: the clipped policy
// loss with a KL term, and the preference loss over pairs of sequences.
//
// A row of logits z predicts one token y: l = z[y] - log sum_j exp(z_j). Both losses
// are functions of the rows' l, so the gradient of a row is one coefficient times
// (one-hot(y) - softmax(z)). Per element that is two exponentials against four to
// eight bytes moved: HBM-bound (without any exponential 4096 rows of 131072 bf16 take 343 us instead
// of 360).
//
// The policy loss reads a row once, keeps it in registers and writes its gradient: 2048 rows of 32000
// bf16 take 49.9 us (rows 44.6 of them, 4.8 TB/s), 4096 of 131072 357 us (354, 5.1 TB/s). The gradient
// of the preference loss needs its whole sequence first, so rows are read twice: 2048 rows of 32000
// take 54.6 us (statistics 19.6, pairs 6, gradient 28.9), 4096 of 50001 fp16 159 us (61 and 97).
//
// The softmax is taken about a maximum in fp32. What is formed once per row or per
// sequence (the sum over the waves, l, the ratio, the sums of l) is formed in fp64: l is
// a difference of numbers much larger than the error that a ratio near its bound may carry.
#include <algorithm>
#include <initializer_list>

#include "row_ops.hpp"

namespace kfac {

constexpr int LT = 256;    // threads of the blocks that hold no row
constexpr int ONE = 1024;  // of a block that is alone
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
  const int64_t y = gp(a.token)[t];
  const bool kept = a.mask ? gp(a.mask)[t] != 0 : true;
  return kept & (y >= 0) & (y < a.vocab);
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

__device__ inline MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == NEG_INF) return {m, a.s + b.s};  // as below
  return {m, a.s * exp(static_cast<double>(a.m) - m) + b.s * exp(static_cast<double>(b.m) - m)};
}
// The lanes' sets as one, in every lane.
__device__ inline MaxSum join_lanes(MaxSum v) {
  const float m = wave_max(v.m);
  // nothing but -inf: no weight, though a NaN stays in the sum
  const double s = m == NEG_INF ? v.s : v.s * exp(static_cast<double>(v.m) - m);
  return {m, wave_add(s)};
}

// A row of any address as groups of 16 bytes: `head` elements up to the first aligned group, `full`
// groups, and the elements behind them. (Groups across two lines cost a tenth of the rate on rows of
// 50001 fp16 elements.) The elements outside the groups, fewer than 2 EV, go one to a thread.
template <class T>
struct Cut {
  static constexpr int EV = Pack<T>::n;
  int first, full;            // element of the first group, groups
  int head, singles, behind;  // elements before the groups, elements outside them, elements in them
  __device__ inline Cut(const KG T* z, int vocab) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(z) / sizeof(T)) & (EV - 1);
    first = head = min(vocab, (EV - off) & (EV - 1));
    full = (vocab - head) / EV;
    behind = full * EV;
    singles = vocab - behind;
  }
  // The groups [b n, b n + n) alone; with the first of them the elements outside the groups.
  __device__ inline Cut part(int b, int n) const {
    Cut c = *this;
    c.first += b * n * EV;
    c.full = max(0, min(full - b * n, n));
    if (b) c.singles = 0;
    return c;
  }
  __device__ inline int64_t group(int g) const { return first + int64_t(g) * EV; }
  __device__ inline bool has_single(int i) const { return i < singles; }
  __device__ inline int single(int i) const { return i < head ? i : behind + i; }
};

// Gradient of a row, coef (one-hot(y) - softmax): -coef softmax(z) everywhere but at y.
template <class T>
struct GradRow {
  typedef typename Pack<T>::vec V;
  static constexpr int EV = Pack<T>::n;
  float m, scale;  // 16-bit types: log2(|coef| / sum); fp32: -coef / sum
  float at_y;
  int y, group_y, place_y;  // the token; its group and place there
  unsigned sign;            // flips the signs of two 16-bit results
  __device__ inline GradRow(const Cut<T>& cut, float m_, double sum, int y_, float z_y, float coef) : m(m_), y(y_) {
    group_y = y < cut.first ? -1 : (y - cut.first) / EV;
    place_y = (y - cut.first) & (EV - 1);
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
    if (g == group_y)
#pragma unroll
      for (int u = 0; u < EV; ++u) w[u] = u == place_y ? static_cast<T>(at_y) : w[u];
    return w;
  }
  __device__ inline T one(float z, int j) const {
    const float w = weight(z);
    return static_cast<T>(j == y ? at_y : sign && sizeof(T) == 2 ? -w : w);
  }
};

// A row over NT threads, C groups of 16 bytes in each thread's registers: all loads are in
// flight at once and the row is read from memory once. Groups past the row hold -inf, which
// weighs nothing; `rest` is the thread's element outside the groups. A group index that no thread
// reaches is skipped by all. C = 0: the row stays in memory and is read again for its gradient.
template <class T, int NT, int C>
struct Row {
  typedef typename Pack<T>::vec V;
  static constexpr int EV = Pack<T>::n;
  V v[C ? C : 1];
  float rest;

  template <bool PAST>
  __device__ inline void load(const Cut<T>& cut, const KG T* z, int tid) {
    const int full = cut.full;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * NT < full) {
#pragma unroll
        for (int u = 0; u < EV; ++u) v[c][u] = static_cast<T>(NEG_INF);
        if (c * NT + tid < full) v[c] = load_pack<PAST, T>(z + cut.group(c * NT + tid));
      }
    rest = cut.has_single(tid) ? static_cast<float>(z[cut.single(tid)]) : NEG_INF;
  }

  // Of the wave's part of the row, in every lane.
  __device__ inline MaxSum wave_stats(const Cut<T>& cut, const KG T* z, int tid) const {
    const int full = cut.full;
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
    } else {  // BATCH groups at a time; a running maximum in each thread, the sum about it in fp64
      constexpr int BATCH = 4;  // with 8 within 2% of it
      float m = rest;
      double s = rest == NEG_INF ? 0.0 : exp_about(rest, rest);
      for (int g0 = tid; g0 < full; g0 += NT * BATCH) {
        V x[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
#pragma unroll
          for (int u = 0; u < EV; ++u) x[b][u] = static_cast<T>(NEG_INF);
          if (g0 + b * NT < full) x[b] = load_pack<false, T>(z + cut.group(g0 + b * NT));
        }
        float top = m;
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
          for (int u = 0; u < EV; ++u) top = fmaxf(top, static_cast<float>(x[b][u]));
        const float at = top == NEG_INF ? 0.f : top;
        if (top != m) s *= exp_about(m, at);
        m = top;
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          v4u raw = __builtin_bit_cast(v4u, x[b]);
          asm("" : "+v"(raw));  // widened again, as above
          const V w = __builtin_bit_cast(V, raw);
          float e = 0;
#pragma unroll
          for (int u = 0; u < EV; ++u) e += exp_about(static_cast<float>(w[u]), at);
          s += e;
        }
      }
      return join_lanes({m, s});
    }
  }

  // An element is read and written by one thread: d may be z.
  template <bool PAST>
  __device__ inline void gradient(const Cut<T>& cut, const GradRow<T>& k, const KG T* z, KG T* d, int tid) const {
    const int full = cut.full;
    if (cut.has_single(tid)) d[cut.single(tid)] = k.one(rest, cut.single(tid));
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * NT + tid < full) {
          const int g = c * NT + tid;
          store_pack<PAST, T>(d + cut.group(g), k.group(v[c], g));
        }
    } else {
      for (int g = tid; g < full; g += NT) {
        const V x = load_pack<false, T>(z + cut.group(g));
        store_pack<PAST, T>(d + cut.group(g), k.group(x, g));
      }
    }
  }
};

template <class T, int NT, bool PAST>
__device__ inline void row_zero(const Cut<T>& cut, KG T* d, int tid) {
  const typename Pack<T>::vec w = {};
  if (cut.has_single(tid)) d[cut.single(tid)] = static_cast<T>(0.f);
  for (int g = tid; g < cut.full; g += NT) store_pack<PAST, T>(d + cut.group(g), w);
}

// A row's block: a wave for a short row (four rows a block, no barrier), else a block.
template <int NT>
constexpr int kRowsPerBlock = NT == 64 ? 4 : 1;
template <int NT>
constexpr int kRowThreads = NT == 64 ? 256 : NT;

// What a wave knows of its row: statistics of its part, and a share of the rows that count.
struct WavePart {
  MaxSum v;
  int n;
};

// The waves' parts as the row's, in the row's first wave.
template <int NT>
__device__ inline WavePart join_waves(WavePart w, WavePart* lds) {
  if constexpr (NT > 64) {
    const int lane = threadIdx.x & 63;
    if (lane == 0) lds[threadIdx.x >> 6] = w;
    __syncthreads();
    if (threadIdx.x < 64) {
      w = lane < NT / 64 ? lds[lane] : WavePart{{NEG_INF, 0.0}, 0};
      w.v = join_lanes(w.v);
      w.n = wave_add(w.n);
    }
  }
  return w;
}

// Rows that count, in gridDim.y slices. By sequence (row_seq given): of each sequence, and per
// row its sequence, -1 where the row does not count; rows outside every sequence get -2. Else: of
// all sequences together.
__global__ void __launch_bounds__(LT) loss_count_kernel(LossRows a, int32_t* __restrict__ row_seq,
                                                        int32_t* __restrict__ count) {
  __shared__ int s[LT / 64];
  const int q = blockIdx.x, slice = blockIdx.y, slices = gridDim.y;
  int r0, r1, n = 0;
  if (row_seq) seq_range(a, q, q + 1, r0, r1);
  else seq_range(a, 0, a.seqs, r0, r1);
  const int per = (r1 - r0 + slices - 1) / slices;
  const int b0 = min(r0 + slice * per, r1), b1 = min(b0 + per, r1);
  for (int t = b0 + threadIdx.x; t < b1; t += LT) {
    const bool counts = row_counts(a, t);
    if (row_seq) row_seq[t] = counts ? q : -1;
    n += counts;
  }
  n = block_add<LT>(n, s);
  if (threadIdx.x == 0) count[q * slices + slice] = n;
  if (row_seq && q == 0 && slice == 0)
    for (int t = threadIdx.x; t < r0; t += LT) row_seq[t] = -2;
  if (row_seq && q == a.seqs - 1 && slice == 0)
    for (int t = r1 + threadIdx.x; t < a.rows; t += LT) row_seq[t] = -2;
}

struct PolicyArgs {
  const float* old_logp;
  const float* ref_logp;  // NULL: no KL term
  const float* advantage;
  float* logp;
  float low, high, kl_coef, grad_scale;
  // what loss_count_kernel left; by sequence both, over all rows `count` alone, and neither where
  // the blocks count for themselves
  const int32_t* row_seq;
  const int32_t* count;
  const int32_t* nonempty;  // the sequences that have a row that counts; NULL: a wave counts them
  int32_t slices;
};

// Weighted surrogate loss, KL and clipped share of a row.
struct PolicyTerms {
  double part, kl, over;
};

enum Place { OUTSIDE, IDLE, COUNTS };  // of a row: in no sequence; in one, not counting; counting

// Place of row t, and its sequence where rows weigh by sequence.
__device__ inline Place row_place(const LossRows& a, const int32_t* row_seq, int t, int& q) {
  const bool counts = row_counts(a, t);
  if (row_seq) {  // offsets that decrease leave rows that no sequence wrote: q may be anything
    q = row_seq[t];
    return q < -1 || q >= a.seqs ? OUTSIDE : q >= 0 && counts ? COUNTS : IDLE;
  }
  int r0, r1;
  seq_range(a, 0, a.seqs, r0, r1);
  return t < r0 || t >= r1 ? OUTSIDE : counts ? COUNTS : IDLE;
}

// A thread's share of the rows that count, for a block that counts for itself.
__device__ inline int own_count(const LossRows& a, int tid, int threads) {
  int r0, r1, n = 0;
  seq_range(a, 0, a.seqs, r0, r1);
  for (int t = r0 + tid; t < r1; t += threads) n += row_counts(a, t);
  return n;
}

// A lane's share of the sequences that have a row that counts.
__device__ inline int nonempty_share(const int32_t* count, int seqs, int slices, int lane, int lanes) {
  int n = 0;
  for (int i = lane; i < seqs; i += lanes) {
    int k = 0;
    for (int j = 0; j < slices; ++j) k |= count[i * slices + j];
    n += k != 0;
  }
  return n;
}
// Of many sequences, for all rows.
__global__ void __launch_bounds__(ONE) loss_nonempty_kernel(const int32_t* __restrict__ count, int seqs, int slices,
                                                            int32_t* __restrict__ out) {
  __shared__ int s[ONE / 64];
  const int n = block_add<ONE>(nonempty_share(count, seqs, slices, threadIdx.x, ONE), s);
  if (threadIdx.x == 0) out[0] = n;
}

// 1 / weight of the rows of sequence q; n: the rows that count, of a block that counted. A wave's work.
__device__ inline double inverse_weight(const LossRows& a, const PolicyArgs& p, int q, int n) {
  const int lane = threadIdx.x & 63;
  if (!p.count) return n;
  if (!p.row_seq) return wave_add(lane < p.slices ? p.count[lane] : 0);
  int own = 0;
  for (int j = 0; j < p.slices; ++j) own += p.count[q * p.slices + j];
  const int full = p.nonempty ? p.nonempty[0] : wave_add(nonempty_share(p.count, a.seqs, p.slices, lane, 64));
  return static_cast<double>(full) * own;
}

// Loss of row t from its softmax, and the coefficient of its gradient; `shown` writes l.
__device__ inline float policy_row(const PolicyArgs& p, int t, float z_y, MaxSum r, double weight, bool shown,
                                   PolicyTerms& out) {
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
    kl = e < __builtin_huge_val() ? e - x : e;  // l of -inf: infinite, not inf - inf
    if (p.kl_coef != 0.f) slope -= p.kl_coef * e;
  }
  if (shown) gp(p.logp)[t] = static_cast<float>(l);
  out = {weight * -(over ? held : free), weight * kl, over ? weight : 0.0};
  return static_cast<float>(p.grad_scale * weight * slope);
}

template <class T, int NT, int C, bool PAST>
__global__ void __launch_bounds__(kRowThreads<NT>) policy_rows_kernel(LossRows a, PolicyArgs p,
                                                                      PolicyTerms* __restrict__ terms) {
  __shared__ WavePart lds[NT / 64];
  __shared__ struct { double s; float m, coef; } row_s;
  const int tid = threadIdx.x & (NT - 1);
  const int t = blockIdx.x * kRowsPerBlock<NT> + (NT == 64 ? threadIdx.x >> 6 : 0);
  if (t >= a.rows) return;
  int q = 0;
  const Place place = row_place(a, p.row_seq, t, q);
  KG T* d = a.dlogits ? gp(static_cast<T*>(a.dlogits)) + t * a.ld_grad : nullptr;
  if (place != COUNTS) {
    if (tid == 0) {
      terms[t] = {0, 0, 0};
      if (place == IDLE) gp(p.logp)[t] = 0.f;
    }
    if (place == IDLE && d) row_zero<T, NT, PAST>(Cut<T>(d, a.vocab), d, tid);
    return;
  }
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  const int y = static_cast<int>(gp(a.token)[t]);
  const float z_y = static_cast<float>(z[y]);
  const Cut<T> cut(z, a.vocab);
  Row<T, NT, C> row;
  row.template load<PAST>(cut, z, tid);
  const int mine = p.count ? 0 : wave_add(own_count(a, tid, NT));
  const WavePart w = join_waves<NT>({row.wave_stats(cut, z, tid), mine}, lds);
  MaxSum r = w.v;
  float coef = 0;
  if (tid < 64) {
    PolicyTerms out;
    coef = policy_row(p, t, z_y, r, 1.0 / inverse_weight(a, p, q, w.n), tid == 0, out);
    if (tid == 0) {
      terms[t] = out;
      if constexpr (NT > 64) {
        row_s.s = r.s;
        row_s.m = r.m;
        row_s.coef = coef;
      }
    }
  }
  if (!d) return;
  if constexpr (NT > 64) {
    __syncthreads();
    r.m = row_s.m;
    r.s = row_s.s;
    coef = row_s.coef;
  }
  row.template gradient<PAST>(cut, GradRow<T>(cut, r.m, r.s, y, z_y, coef), z, d, tid);
}

// A block's sum of terms, in its first thread.
template <int NT>
__device__ inline PolicyTerms block_terms(const PolicyTerms* terms, int r0, int r1) {
  __shared__ PolicyTerms lds[NT / 64];
  PolicyTerms v = {0, 0, 0};
#pragma unroll 4
  for (int t = r0 + threadIdx.x; t < r1; t += NT)
    v = {v.part + terms[t].part, v.kl + terms[t].kl, v.over + terms[t].over};
  v = {wave_add(v.part), wave_add(v.kl), wave_add(v.over)};
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x < 64) {
    v = threadIdx.x < NT / 64 ? lds[threadIdx.x] : PolicyTerms{0, 0, 0};
    v = {wave_add(v.part), wave_add(v.kl), wave_add(v.over)};
  }
  return v;
}

// Many rows, beyond FEW_TERMS: TERMS of them to one. (A call of 6000 rows of 200 takes 16.5 us without
// this launch and 18.8 with it, 20000 rows 31.5 and 29.7, 200000 rows of 64 216 and 172.)
constexpr int TERMS = 2048, FEW_TERMS = 16384;
__global__ void __launch_bounds__(LT) policy_terms_kernel(const PolicyTerms* __restrict__ terms, int rows,
                                                          PolicyTerms* __restrict__ out) {
  const int r0 = blockIdx.x * TERMS;
  const PolicyTerms v = block_terms<LT>(terms, r0, min(rows, r0 + TERMS));
  if (threadIdx.x == 0) out[blockIdx.x] = v;
}

// The loss, its surrogate part, the mean KL, the clipped share.
__device__ inline void policy_stats(PolicyTerms v, float kl_coef, float* stats) {
  gp(stats)[0] = static_cast<float>(kl_coef != 0.f ? v.part + kl_coef * v.kl : v.part);
  gp(stats)[1] = static_cast<float>(v.part);
  gp(stats)[2] = static_cast<float>(v.kl);
  gp(stats)[3] = static_cast<float>(v.over);
}

// One block; of 2048 rows it takes 4.5 us, about the launch.
constexpr int FT = 512;
__global__ void __launch_bounds__(FT) policy_finish_kernel(const PolicyTerms* __restrict__ terms, int rows,
                                                           float kl_coef, float* stats) {
  const PolicyTerms v = block_terms<FT>(terms, 0, rows);
  if (threadIdx.x == 0) policy_stats(v, kl_coef, stats);
}

// Few long rows, which would leave most of the chip idle: blocks for the parts of a row, then blocks
// that join the parts, each for the gradient of a piece of its row, and one for all rows' results. A
// call has at most 64 rows, a row at most 64 parts: a lane each. Latency-bound: 4 rows of 50001 fp16
// take 4.2 and 5.0 us in the kernels, 11.7 a call.
constexpr int SPLIT = 64, SPLIT_C = 4, SPLIT_GROUPS = LT * SPLIT_C;

template <class T>
__global__ void __launch_bounds__(LT) policy_part_kernel(LossRows a, MaxSum* __restrict__ part,
                                                         float* __restrict__ row_z) {
  __shared__ WavePart lds[LT / 64];
  const int t = blockIdx.y;
  int q;
  if (row_place(a, nullptr, t, q) != COUNTS) return;
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  const Cut<T> cut = Cut<T>(z, a.vocab).part(blockIdx.x, SPLIT_GROUPS);
  Row<T, LT, SPLIT_C> row;
  row.template load<false>(cut, z, threadIdx.x);
  const WavePart w = join_waves<LT>({row.wave_stats(cut, z, threadIdx.x), 0}, lds);
  if (threadIdx.x == 0) part[t * gridDim.x + blockIdx.x] = w.v;
  // the token's logit, which the gradient may overwrite before every block has read it
  if (threadIdx.x == 0 && blockIdx.x == 0) row_z[t] = static_cast<float>(z[gp(a.token)[t]]);
}

template <class T>
__global__ void __launch_bounds__(LT) policy_join_kernel(LossRows a, PolicyArgs p, const MaxSum* __restrict__ part,
                                                         const float* __restrict__ row_z, int parts, float* stats) {
  const int lane = threadIdx.x & 63;
  const double weight = 1.0 / wave_add(own_count(a, lane, 64));
  int q;
  if (blockIdx.y == 0) {  // the results, a lane a row
    if (blockIdx.x || threadIdx.x >= 64) return;
    PolicyTerms v = {0, 0, 0};
    const Place place = lane < a.rows ? row_place(a, nullptr, lane, q) : OUTSIDE;
    if (place == IDLE) gp(p.logp)[lane] = 0.f;
    if (place == COUNTS) {
      MaxSum r = part[lane * parts];
      for (int i = 1; i < parts; ++i) r = join(r, part[lane * parts + i]);
      policy_row(p, lane, row_z[lane], r, weight, true, v);
    }
    v = {wave_add(v.part), wave_add(v.kl), wave_add(v.over)};
    if (lane == 0) policy_stats(v, p.kl_coef, stats);
    return;
  }
  const int t = blockIdx.y - 1;
  const Place place = row_place(a, nullptr, t, q);
  if (place == OUTSIDE) return;
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  KG T* d = gp(static_cast<T*>(a.dlogits)) + t * a.ld_grad;
  const Cut<T> cut = Cut<T>(z, a.vocab).part(blockIdx.x, SPLIT_GROUPS);
  if (place == IDLE) {
    row_zero<T, LT, false>(cut, d, threadIdx.x);
    return;
  }
  const int y = static_cast<int>(gp(a.token)[t]);
  const float z_y = row_z[t];
  Row<T, LT, SPLIT_C> row;
  row.template load<false>(cut, z, threadIdx.x);
  const MaxSum r = join_lanes(lane < parts ? part[t * parts + lane] : MaxSum{NEG_INF, 0.0});
  PolicyTerms unused;
  const float coef = policy_row(p, t, z_y, r, weight, false, unused);
  row.template gradient<false>(cut, GradRow<T>(cut, r.m, r.s, y, z_y, coef), z, d, threadIdx.x);
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
  __shared__ WavePart lds[NT / 64];
  const int tid = threadIdx.x & (NT - 1);
  const int t = blockIdx.x * kRowsPerBlock<NT> + (NT == 64 ? threadIdx.x >> 6 : 0);
  int q;
  const Place place = t < a.rows ? row_place(a, nullptr, t, q) : OUTSIDE;
  if (place != COUNTS) {
    if (place == IDLE && tid == 0) row_logp[t] = 0;
    return;
  }
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  const float z_y = static_cast<float>(z[gp(a.token)[t]]);
  const Cut<T> cut(z, a.vocab);
  Row<T, NT, C> row;
  row.template load<false>(cut, z, tid);
  const MaxSum r = join_waves<NT>({row.wave_stats(cut, z, tid), 0}, lds).v;
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

// Pair i from its sequences' sums of l: the margin, its share of the loss, and what its gradient
// takes: the coefficient of a row of the preferred sequence. `shown` writes the results.
__device__ inline float pref_pair(const PrefArgs& p, int i, double chosen, double other, bool shown, double& loss) {
  const double rc = p.ref_logp ? gp(p.ref_logp)[i] : 0.f, rr = p.ref_logp ? gp(p.ref_logp)[i + p.pairs] : 0.f;
  const double x = p.beta * ((chosen - rc) - (other - rr)), e = p.smooth;
  const double t = exp(-fabs(x)), both = log1p(t);
  const double below = fmax(-x, 0.0) + both, above = fmax(x, 0.0) + both;  // log(1 + exp(-x)), log(1 + exp(x))
  const double miss = (x > 0 ? t : 1.0) / (1.0 + t);                       // 1 / (1 + exp(x))
  // either may be infinite, and has no part in the loss where its share is 0
  loss = ((e < 1 ? (1 - e) * below : 0.0) + (e > 0 ? e * above : 0.0)) / p.pairs;
  if (shown) {
    gp(p.margin)[i] = static_cast<float>(x);
    gp(p.seq_logp)[i] = static_cast<float>(chosen);
    gp(p.seq_logp)[i + p.pairs] = static_cast<float>(other);
  }
  return static_cast<float>(p.grad_scale * (e - miss) * p.beta / p.pairs);
}

// Sum of l over a sequence by one wave, the `part`th of `parts`.
__device__ inline double sequence_sum(const LossRows& a, int q, const double* row_logp, int part = 0, int parts = 1) {
  int r0, r1;
  seq_range(a, q, q + 1, r0, r1);
  double v = 0;
#pragma unroll 4
  for (int t = r0 + 64 * part + static_cast<int>(threadIdx.x & 63); t < r1; t += 64 * parts) v += gp(row_logp)[t];
  return wave_add(v);
}

// W waves a sequence, so PAIRS = 8 / W pairs a block: the sums of l, the pair's results, and for
// each row the coefficient of its gradient. part: a block's share of the loss.
constexpr int PAIR_WAVES = ONE / 64;
__global__ void __launch_bounds__(ONE) pref_pairs_kernel(LossRows a, PrefArgs p, const double* __restrict__ row_logp,
                                                         float* __restrict__ row_coef, double* __restrict__ part, int W) {
  __shared__ double sum_s[PAIR_WAVES], loss_s[PAIR_WAVES];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int seq = wave / W, share = wave % W;  // of the block's sequences; of the sequence's waves
  const int local = seq >> 1, side = seq & 1;  // side 1: the other of the pair
  const int i = blockIdx.x * (PAIR_WAVES / 2 / W) + local;
  const bool here = i < p.pairs;
  if (here) {
    const double v = sequence_sum(a, i + side * p.pairs, row_logp, share, W);
    if (lane == 0) sum_s[wave] = v;
  }
  __syncthreads();
  double loss = 0;
  if (here) {
    double sum[2] = {0, 0};
    for (int k = 0; k < 2; ++k)
      for (int w = 0; w < W; ++w) sum[k] += sum_s[(2 * local + k) * W + w];
    const float c = pref_pair(p, i, sum[0], sum[1], side == 0 && share == 0 && lane == 0, loss);
    int r0, r1;
    seq_range(a, i + side * p.pairs, i + side * p.pairs + 1, r0, r1);
    for (int t = r0 + 64 * share + lane; t < r1; t += 64 * W) row_coef[t] = side ? -c : c;
  }
  if (lane == 0) loss_s[wave] = side == 0 && share == 0 ? loss : 0.0;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0;
    for (int k = 0; k < PAIR_WAVES; ++k) total += loss_s[k];
    if (gridDim.x == 1) gp(p.loss)[0] = static_cast<float>(total);
    else part[blockIdx.x] = total;
  }
}

// The loss from the shares of n blocks, by one block.
__device__ inline void pref_total(const double* part, int n, float* loss) {
  __shared__ double s[LT / 64];
  double v = 0;
  for (int i = threadIdx.x; i < n; i += LT) v += gp(part)[i];
  v = block_add<LT>(v, s);
  if (threadIdx.x == 0) gp(loss)[0] = static_cast<float>(v);
}
__global__ void __launch_bounds__(LT) pref_finish_kernel(const double* __restrict__ part, int n, float* loss) {
  pref_total(part, n, loss);
}

// Coefficient of row t's gradient, formed by the wave that needs it (at most 32 sequences).
__device__ inline float row_coefficient(const LossRows& a, const PrefArgs& p, int t, const double* row_logp) {
  const int lane = threadIdx.x & 63;
  // the last sequence that begins at or before t
  const int q = __popcll(__ballot(lane > 0 && lane < a.seqs && gp(a.begin)[lane] <= t));
  const int side = q >= p.pairs, i = q - side * p.pairs;
  double loss;
  const float c =
      pref_pair(p, i, sequence_sum(a, i, row_logp), sequence_sum(a, i + p.pairs, row_logp), false, loss);
  return side ? -c : c;
}

// The results of all pairs by one block, a wave a pair.
__device__ inline void pair_results(const LossRows& a, const PrefArgs& p, const double* row_logp) {
  __shared__ double loss_s[LT / 64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  double loss = 0;
  for (int i = wave; i < p.pairs; i += LT / 64) {
    double share;
    const double chosen = sequence_sum(a, i, row_logp), other = sequence_sum(a, i + p.pairs, row_logp);
    pref_pair(p, i, chosen, other, lane == 0, share);
    loss += share;
  }
  if (lane == 0) loss_s[wave] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < LT / 64; ++w) loss += loss_s[w];
    gp(p.loss)[0] = static_cast<float>(loss);
  }
}

// Elementwise over the rows below `end`, last rows first: what pref_rows_kernel read last is what the
// caches still hold. NT threads take a row, or U groups of 16 bytes each of a longer one (a wave a short
// row, four rows a block: 32768 rows of 250 groups take 63.3 us a call so and 73.0 with a block each; U
// of 2: 2048 rows of 4000 groups 57.0 us, with 4 58.0), and end with their stores: no loop over rows,
// which would wait for them.
// ALONE: no pref_pairs_kernel came before; every row's coefficient is formed here, and by one block
// more in y the pairs' results. Else, with parts, one block more in y adds up the loss from them, which
// saves a launch: 411 rows of 824 fp32 in 32 pairs take 15.8 us instead of 18.9. Not past the caches, where
// the choice cost 4096 rows of 50001 172 us instead of 165.
template <class T, int NT, int U, bool PAST, bool ALONE>
__global__ void __launch_bounds__(LT) pref_grad_kernel(LossRows a, PrefArgs p, const RowStat* __restrict__ row_stat,
                                                       const float* __restrict__ row_coef,
                                                       const double* __restrict__ row_logp,
                                                       const double* __restrict__ part, int parts, int end) {
  int by = blockIdx.y;
  if (ALONE || (!PAST && parts)) {
    if (by == 0) {
      if (blockIdx.x) return;
      if constexpr (ALONE) pair_results(a, p, row_logp);
      else pref_total(part, parts, p.loss);
      return;
    }
    --by;
  }
  const int tid = threadIdx.x & (NT - 1);
  const int t = end - 1 - (by * kRowsPerBlock<NT> + (NT == 64 ? threadIdx.x >> 6 : 0));
  int q;
  const Place place = t >= 0 ? row_place(a, nullptr, t, q) : OUTSIDE;
  if (place == OUTSIDE) return;
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  KG T* d = gp(static_cast<T*>(a.dlogits)) + t * a.ld_grad;
  const Cut<T> cut = Cut<T>(z, a.vocab).part(blockIdx.x, NT * U);
  if (place == IDLE) {
    row_zero<T, NT, PAST>(cut, d, tid);
    return;
  }
  Row<T, NT, U> row;
  row.template load<true>(cut, z, tid);
  const RowStat r = row_stat[t];
  const float coef = ALONE ? row_coefficient(a, p, t, row_logp) : row_coef[t];
  const GradRow<T> k(cut, r.m, r.s, static_cast<int>(gp(a.token)[t]), r.z_y, coef);
  row.template gradient<PAST>(cut, k, z, d, tid);
}

}  // namespace kfac

using namespace kfac;

static kfac_status rows_validate(int32_t rows, int32_t vocab, int32_t seqs) {
  if (rows < 0) return fail(KFAC_ERR_INVALID, "rows must be >= 0");
  // a launch may have 2^32 threads, and a row 1024 of them
  if (rows >= (1 << 22)) return fail(KFAC_ERR_UNSUPPORTED, "%d rows: more than one call takes", rows);
  if (vocab < 1 || vocab > (1 << 30)) return fail(KFAC_ERR_INVALID, "vocab = %d out of range", vocab);
  if (seqs < 0 || seqs > (1 << 22)) return fail(KFAC_ERR_INVALID, "%d sequences: out of range", seqs);
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

// Bytes of a call's buffer; none where it is NULL.
struct Bytes {
  const void* p;
  int64_t n;
};
// No result may share bytes with an input: blocks that write it and blocks that read it run at
// once. (The gradient and the logits are rows_check's.)
static kfac_status check_apart(std::initializer_list<Bytes> results, std::initializer_list<Bytes> inputs) {
  for (const Bytes& r : results)
    for (const Bytes& i : inputs) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(r.p), y = reinterpret_cast<uintptr_t>(i.p);
      if (x && y && r.n && i.n && x < y + i.n && y < x + r.n) return fail(KFAC_ERR_INVALID, "a result overlaps an input");
    }
  return KFAC_OK;
}
static Bytes rows_of(const void* p, const LossRows& a, int64_t ld, kfac_dtype dtype) {
  return {p, a.rows ? ((a.rows - 1) * ld + a.vocab) * (dtype == KFAC_F32 ? 4 : 2) : 0};
}

// Nor with another result or the workspace, which are written at once too; `written` holds all of
// them but the gradient, of which its rows count and not what lies between them.
static kfac_status check_written(const LossRows& a, kfac_dtype dtype, std::initializer_list<Bytes> written) {
  const int64_t size = dtype == KFAC_F32 ? 4 : 2, pitch = a.ld_grad * size, width = a.vocab * size;
  const uintptr_t d = reinterpret_cast<uintptr_t>(a.dlogits);
  for (auto x = written.begin(); x != written.end(); ++x) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(x->p), e = b + x->n;
    if (!b || !x->n) continue;
    for (auto y = written.begin(); y != x; ++y) {
      const uintptr_t o = reinterpret_cast<uintptr_t>(y->p);
      if (o && y->n && b < o + y->n && o < e) return fail(KFAC_ERR_INVALID, "results overlap each other or the workspace");
    }
    if (!d || !a.rows || e <= d) continue;
    const uintptr_t row = b > d ? (b - d) / pitch : 0;  // the first that may hold one of its bytes, or the next
    for (uintptr_t r = row; r < uintptr_t(a.rows) && r <= row + 1; ++r)
      if (b < d + r * pitch + width && d + r * pitch < e)
        return fail(KFAC_ERR_INVALID, "dlogits overlaps a result or the workspace");
  }
  return KFAC_OK;
}

// LAUNCH(type) for the type of a code.
#define KFAC_BY_TYPE(dtype, LAUNCH)              \
  do {                                           \
    if ((dtype) == KFAC_F32) { LAUNCH(float) }   \
    else if ((dtype) == KFAC_BF16) { LAUNCH(__bf16) } \
    else { LAUNCH(_Float16) }                    \
  } while (0)

// LAUNCH(T, NT, C) for a row length: C groups of 16 bytes, four registers each, in NT threads. Policy
// calls, in us:
//    250 groups, 32768 rows:  58.5 in   64 x 4 (four rows a block, no barrier),  99.5 in  256 x 4
//   1000 groups, 16384 rows: 103   in  256 x 4,                                 107   in  256 x 8
//   2000 groups,  8192 rows: 102   in  256 x 8,                                 108   in  512 x 8
//   4000 groups,  2048 rows:  50.3 in  512 x 8,       52.4 in 256 x 16,  51.9 in 1024 x 4
//   6250 groups,  4096 rows: 173   in 512 x 16,                                 192   in 1024 x 8
//  16384 groups,  4096 rows: 433.5 in 1024 x 16,                                435.3 in 1024 x 19
// A row that waits in its registers for its gradient (`keep`) may have 19 groups a thread, the most that
// leave no spills under the 128 registers of a 1024-thread block: 4096 rows of 16384 groups take 429 us
// so, 470 if they stay in memory (no row masked). Rows without a gradient stay there from 8192 groups on,
// two blocks on a CU instead of one: 1453 rows of 11803 groups 63.9 us instead of 83.4, 1453 of 16384
// 78.3 instead of 96.9; in blocks of 512 threads 62.7 and 81.5. Longer rows stay in memory.
#define KFAC_SHORT_ROWS(T, LAUNCH)                   \
  if (groups_ <= 64 * 4) { LAUNCH(T, 64, 4) }        \
  else if (groups_ <= 256 * 4) { LAUNCH(T, 256, 4) } \
  else if (groups_ <= 256 * 8) { LAUNCH(T, 256, 8) } \
  else if (groups_ <= 512 * 8) { LAUNCH(T, 512, 8) } \
  else if (groups_ <= 512 * 16) { LAUNCH(T, 512, 16) }
#define KFAC_BY_ROW(T, vocab, keep, LAUNCH)                          \
  do {                                                               \
    const int groups_ = (vocab) / Pack<T>::n;                        \
    KFAC_SHORT_ROWS(T, LAUNCH)                                       \
    else if ((keep) && groups_ <= 1024 * 16) { LAUNCH(T, 1024, 16) } \
    else if ((keep) && groups_ <= 1024 * 19) { LAUNCH(T, 1024, 19) } \
    else { LAUNCH(T, 1024, 0) }                                      \
  } while (0)
#define KFAC_BY_STATS(T, vocab, LAUNCH)       \
  do {                                        \
    const int groups_ = (vocab) / Pack<T>::n; \
    KFAC_SHORT_ROWS(T, LAUNCH)                \
    else { LAUNCH(T, 1024, 0) }               \
  } while (0)

static int64_t row_bytes(int32_t rows, int32_t vocab, kfac_dtype dtype) {
  return int64_t(rows) * vocab * (dtype == KFAC_F32 ? 4 : 2);
}
// Rows of more than this pass the caches by where they are read or written once. What is dirty in
// the 256 MB last-level cache is written back later at the expense of what is read then: 131 MB of
// rows take 50 us instead of 56 (policy) and 53.7 instead of 63.6 (preference). The first pass of the
// preference loss stays in the caches for the second: 410 MB take 166 us instead of 186.
constexpr int64_t STORE_PAST = int64_t(64) << 20;

// A count of rows: by sequence in 256-row slices, up to 16; over all rows in up to 64.
static int count_slices(int32_t rows, int32_t seqs, bool by_seq) {
  const int64_t n = rows / (int64_t(by_seq ? seqs : 1) * LT), most = by_seq ? 16 : 64;
  return n < 1 ? 1 : n > most ? static_cast<int>(most) : static_cast<int>(n);
}

// Steps over counts that the rows of a call by sequence take for themselves.
constexpr int64_t OWN_STEPS = 200000;

// Rows of more groups than this are cut into parts where they are few: one row of 131072 bf16 takes
// 11.9 us against 20.4 whole, 16 rows of 32000 25.1 against 27.5 when the caller waits, 64 rows of 131072
// 18.4 against 24.0; at 9000 elements, 1125 groups, both take the same.
constexpr int SPLIT_FROM = 1024;

struct PolicyWs {
  int32_t *row_seq, *count, *nonempty;
  PolicyTerms *terms, *sums;
  MaxSum* part;
  float* row_z;
  size_t bytes;
};
static PolicyWs policy_ws(void* ws, int32_t rows, int32_t seqs) {
  Carver cv(ws);
  PolicyWs w;
  w.row_seq = cv.take<int32_t>(rows);
  w.count = cv.take<int32_t>(std::max<size_t>(64, size_t(seqs) * (seqs ? count_slices(rows, seqs, true) : 0)));
  w.nonempty = cv.take<int32_t>(1);
  w.terms = cv.take<PolicyTerms>(rows);
  w.sums = cv.take<PolicyTerms>(rows / TERMS + 1);
  w.part = cv.take<MaxSum>(size_t(std::min(rows, SPLIT)) * SPLIT);
  w.row_z = cv.take<float>(SPLIT);
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

static kfac_status launch_finish(const PolicyWs& w, int32_t rows, float kl_coef, float* stats, hipStream_t s) {
  const PolicyTerms* terms = w.terms;
  if (rows > FEW_TERMS) {
    const int blocks = (rows - 1) / TERMS + 1;
    KFAC_LAUNCH(K_POLICY_TERMS, policy_terms_kernel, dim3(blocks), dim3(LT), 0, s, w.terms, rows, w.sums);
    KFAC_CHECK_LAUNCH("policy_terms_kernel");
    terms = w.sums;
    rows = blocks;
  }
  KFAC_LAUNCH(K_POLICY_FINISH, policy_finish_kernel, dim3(1), dim3(FT), 0, s, terms, rows, kl_coef, stats);
  KFAC_CHECK_LAUNCH("policy_finish_kernel");
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
    const int64_t n = rows;
    const Bytes in_z = rows_of(logits, a, ld, dtype), in_token = {token, 8 * n}, in_mask = {mask, n},
                in_begin = {seq_begin, 4 * (int64_t(seqs) + 1)}, in_old = {old_logp, 4 * n},
                in_ref = {ref_logp, 4 * n}, in_adv = {advantage, 4 * n};
    if ((st = check_apart({{logp, 4 * n}, {stats, 16}}, {in_z, in_token, in_mask, in_begin, in_old, in_ref, in_adv})) ||
        (st = check_apart({rows_of(dlogits, a, ld_grad, dtype)},
                          {in_token, in_mask, in_begin, in_old, in_ref, in_adv})))
      return st;
  }
  if ((st = check_device())) return st;
  const PolicyWs w = policy_ws(workspace, rows, seqs);
  if ((st = check_workspace(workspace, ws_bytes, w.bytes))) return st;
  if ((st = check_written(a, dtype, {{logp, 4 * int64_t(rows)}, {stats, 16}, {workspace, int64_t(w.bytes)}}))) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  PolicyArgs p = {old_logp, ref_logp, advantage, logp, clip_low, clip_high, kl_coef, grad_scale, nullptr, nullptr, nullptr, 0};
  const bool by_seq = by_sequence && seqs > 1;  // the mean over one sequence is the mean over its rows
  if (rows == 0) return launch_finish(w, rows, kl_coef, stats, s);
  const int64_t groups = vocab / (dtype == KFAC_F32 ? 4 : 8), parts = groups / SPLIT_GROUPS + 1;
  if (!by_seq && rows <= SPLIT && parts <= SPLIT && groups > SPLIT_FROM) {
#define KFAC_TYPED(T)                                                                                            \
  KFAC_LAUNCH(K_POLICY_PART, policy_part_kernel<T>, dim3(parts, rows), dim3(LT), 0, s, a, w.part, w.row_z);      \
  KFAC_CHECK_LAUNCH("policy_part_kernel");                                                                       \
  KFAC_LAUNCH(K_POLICY_JOIN, policy_join_kernel<T>, dlogits ? dim3(parts, rows + 1) : dim3(1, 1), dim3(LT), 0, s, a, \
              p, w.part, w.row_z, static_cast<int>(parts), stats);
    KFAC_BY_TYPE(dtype, KFAC_TYPED);
#undef KFAC_TYPED
    KFAC_CHECK_LAUNCH("policy_join_kernel");
    return KFAC_OK;
  }
  // Where a row's threads have one row each to look at (a wave up to four) they count for themselves,
  // behind the loads of their own row, which saves the launch (4.6 us); with four each, 4096 rows of
  // 131072 took 387 us instead of 360.
  int row_threads = 0;
#define KFAC_THREADS(T, NT, C) row_threads = NT;
#define KFAC_TYPED(T) KFAC_BY_ROW(T, vocab, dlogits, KFAC_THREADS);
  KFAC_BY_TYPE(dtype, KFAC_TYPED);
#undef KFAC_TYPED
#undef KFAC_THREADS
  if (by_seq || rows > std::max(row_threads, 256)) {
    p.row_seq = by_seq ? w.row_seq : nullptr;
    p.count = w.count;
    p.slices = count_slices(rows, seqs, by_seq);
    KFAC_LAUNCH(K_LOSS_COUNT, loss_count_kernel, dim3(by_seq ? seqs : 1, p.slices), dim3(LT), 0, s, a,
                by_seq ? w.row_seq : nullptr, w.count);
    KFAC_CHECK_LAUNCH("loss_count_kernel");
    // A wave looks for the sequences that hold its row's weight itself, `steps` counts behind one another, or they
    // are counted before: 300 sequences over 8192 rows of 1000 take 22.1 us without this launch and 23.2 with
    // it, 2000 sequences 26.7 and 24.6. Every row repeats the steps: rows of 64 bf16 take 28.4 us without it and
    // 29.5 with it at 20000 rows in 16 sequences (4 steps), 35.3 and 29.0 in 1000 (16 steps), 72.2 and 66.0 at 60000
    // rows in two (16 steps), 3657 and 894 at 10^6 in 300 (65 steps).
    const int64_t steps = int64_t((seqs + 63) / 64) * p.slices;
    if (by_seq && (seqs > 1024 || rows * steps > OWN_STEPS)) {
      p.nonempty = w.nonempty;
      KFAC_LAUNCH(K_LOSS_NONEMPTY, loss_nonempty_kernel, dim3(1), dim3(ONE), 0, s, w.count, seqs, p.slices, w.nonempty);
      KFAC_CHECK_LAUNCH("loss_nonempty_kernel");
    }
  }
  const bool past = row_bytes(rows, vocab, dtype) > STORE_PAST;
#define KFAC_ROWS(T, NT, C)                                                                                      \
  const unsigned grid = (rows - 1) / kRowsPerBlock<NT> + 1;                                                      \
  if (past) {                                                                                                    \
    KFAC_LAUNCH(K_POLICY_ROWS, (policy_rows_kernel<T, NT, C, true>), dim3(grid), dim3(kRowThreads<NT>), 0, s, a, \
                p, w.terms);                                                                                     \
  } else {                                                                                                       \
    KFAC_LAUNCH(K_POLICY_ROWS, (policy_rows_kernel<T, NT, C, false>), dim3(grid), dim3(kRowThreads<NT>), 0, s, a, \
                p, w.terms);                                                                                     \
  }
#define KFAC_TYPED(T) KFAC_BY_ROW(T, vocab, dlogits, KFAC_ROWS);
  KFAC_BY_TYPE(dtype, KFAC_TYPED);
#undef KFAC_TYPED
#undef KFAC_ROWS
  KFAC_CHECK_LAUNCH("policy_rows_kernel");
  return launch_finish(w, rows, kl_coef, stats, s);
}

// Up to here the gradient's blocks wait less for their sums than the launch of pref_pairs_kernel takes
// (1000 rows of 1000 in fp32: 14.6 against 16.8 us; 300 of 32000: 25.2 against 23.5). Each row's wave adds up
// its whole pair, however the pairs share the rows, so their number is bounded too: rows of 2 to 100
// elements in one pair take 12.6 against 15.7 us at 2000 rows, 13.7 against 15.7 at 3000, 17.3 against 16.5 at
// 4000, 55 against 18 at 10000; in 16 pairs of which one has nearly all rows 15.0 against 16.0 at 3000, 18.6
// against 18.6 at 4000, 57 against 32 at 10000.
constexpr int64_t ALONE_BYTES = int64_t(8) << 20;
constexpr int ALONE_ROWS = 3000;

struct PrefWs {
  RowStat* stat;
  double *logp, *part;
  float* coef;
  size_t bytes;
};
// Waves of a sequence: about four rows a lane, while the pairs fit in one block; with more pairs
// than that, or sequences longer than 16 rows a lane, several blocks and a launch to add their losses.
// (One wave each: two sequences over 8192 rows of 1000 take 27.2 us a call instead of 21.3, eight over
// 60000 rows of 200 71.9 instead of 53.3.)
static int sequence_waves(int32_t rows, int32_t pairs) {
  const int64_t per = pairs < 1 ? 1 : rows / (2 * int64_t(pairs)) + 1;
  int w = 1;
  while (w < PAIR_WAVES / 2 && per > 256 * w && (pairs * w < PAIR_WAVES / 2 || per > 1024 * w)) w *= 2;
  return w;
}
static int pair_blocks(int32_t rows, int32_t pairs) {
  const int each = PAIR_WAVES / 2 / sequence_waves(rows, pairs);
  return pairs < 1 ? 1 : (pairs - 1) / each + 1;
}

static PrefWs pref_ws(void* ws, int32_t rows, int32_t pairs) {
  Carver cv(ws);
  PrefWs w;
  w.stat = cv.take<RowStat>(rows);
  w.logp = cv.take<double>(rows);
  w.part = cv.take<double>(pair_blocks(rows, pairs));
  w.coef = cv.take<float>(rows);
  w.bytes = cv.used;
  return w;
}

extern "C" kfac_status kfac_preference_loss_workspace(int32_t rows, int32_t vocab, int32_t pairs, size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  if (pairs < 0 || pairs > (1 << 21)) return fail(KFAC_ERR_INVALID, "%d pairs: out of range", pairs);
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
  if (pairs < 0 || pairs > (1 << 21)) return fail(KFAC_ERR_INVALID, "%d pairs: out of range", pairs);
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
    const int64_t n = rows, seqs = 2 * int64_t(pairs);
    const Bytes in_z = rows_of(logits, a, ld, dtype), in_token = {token, 8 * n}, in_mask = {mask, n},
                in_begin = {seq_begin, 4 * (seqs + 1)}, in_ref = {ref_logp, 4 * seqs};
    if ((st = check_apart({{seq_logp, 4 * seqs}, {margin, 2 * seqs}, {loss, 4}},
                          {in_z, in_token, in_mask, in_begin, in_ref})) ||
        (st = check_apart({rows_of(dlogits, a, ld_grad, dtype)}, {in_token, in_mask, in_begin, in_ref})))
      return st;
  }
  if ((st = check_device())) return st;
  const PrefWs w = pref_ws(workspace, rows, pairs);
  if ((st = check_workspace(workspace, ws_bytes, w.bytes))) return st;
  const int64_t n = pairs;
  if ((st = check_written(a, dtype, {{seq_logp, 8 * n}, {margin, 4 * n}, {loss, 4}, {workspace, int64_t(w.bytes)}})))
    return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const PrefArgs p = {ref_logp, seq_logp, margin, loss, beta, label_smoothing, grad_scale, pairs};
  const bool any = rows > 0 && pairs > 0;
  const bool store_past = row_bytes(rows, vocab, dtype) > STORE_PAST;
  if (any) {
#define KFAC_ROWS(T, NT, C)                                                                        \
  KFAC_LAUNCH(K_PREF_ROWS, (pref_rows_kernel<T, NT, C>), dim3((rows - 1) / kRowsPerBlock<NT> + 1), \
              dim3(kRowThreads<NT>), 0, s, a, w.stat, w.logp);
#define KFAC_TYPED(T) KFAC_BY_STATS(T, vocab, KFAC_ROWS);
    KFAC_BY_TYPE(dtype, KFAC_TYPED);
#undef KFAC_TYPED
#undef KFAC_ROWS
    KFAC_CHECK_LAUNCH("pref_rows_kernel");
  }
  // A small call with few pairs: the gradient's blocks form their own coefficients, each from the l of
  // one pair, and one of them the pairs' results.
  const bool alone =
      any && dlogits && pairs <= 16 && rows <= ALONE_ROWS && row_bytes(rows, vocab, dtype) <= ALONE_BYTES;
  int parts = 0;  // of the loss, where several blocks have a share each
  if (!alone) {
    const int blocks = pair_blocks(rows, pairs);
    KFAC_LAUNCH(K_PREF_PAIRS, pref_pairs_kernel, dim3(blocks), dim3(ONE), 0, s, a, p, w.logp, w.coef, w.part,
                sequence_waves(rows, pairs));
    KFAC_CHECK_LAUNCH("pref_pairs_kernel");
    if (blocks > 1) parts = blocks;
    if (parts && (store_past || !any || !dlogits)) {
      KFAC_LAUNCH(K_PREF_FINISH, pref_finish_kernel, dim3(1), dim3(LT), 0, s, w.part, parts, loss);
      KFAC_CHECK_LAUNCH("pref_finish_kernel");
      parts = 0;
    }
  }
  if (any && dlogits) {
    const bool waves = vocab / (dtype == KFAC_F32 ? 4 : 8) <= 64 * 4;  // a wave holds a row
    const int most = 65534 * (waves ? 4 : 1);                         // rows of a grid
    for (int32_t end = rows; end > 0; end -= most, parts = 0) {
      const unsigned blocks = (std::min(end, most) - 1) / (waves ? 4 : 1) + 1 + (alone || parts);
#define KFAC_GRAD(T, NT, U, PAST, ALONE)                                                                     \
  KFAC_LAUNCH(K_PREF_GRAD, (pref_grad_kernel<T, NT, U, PAST, ALONE>),                                        \
              dim3((vocab / Pack<T>::n) / (NT * U) + 1, blocks), dim3(LT), 0, s, a, p, w.stat, w.coef, w.logp, \
              w.part, parts, end);
#define KFAC_ROWS(T, NT, U)                                    \
  if (alone) { KFAC_GRAD(T, NT, U, false, true) }              \
  else if (store_past) { KFAC_GRAD(T, NT, U, true, false) }    \
  else { KFAC_GRAD(T, NT, U, false, false) }
#define KFAC_TYPED(T)                     \
  if (waves) { KFAC_ROWS(T, 64, 4) }      \
  else { KFAC_ROWS(T, 256, 2) }
      KFAC_BY_TYPE(dtype, KFAC_TYPED);
#undef KFAC_TYPED
#undef KFAC_ROWS
#undef KFAC_GRAD
      KFAC_CHECK_LAUNCH("pref_grad_kernel");
    }
  }
  return KFAC_OK;
}
