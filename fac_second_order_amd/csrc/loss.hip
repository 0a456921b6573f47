// Losses over a model's logits with their gradient in the logits: the clipped policy
// loss with a KL term, and the preference loss over pairs of sequences.
//
// A row of logits z predicts one token y: l = z[y] - log sum_j exp(z_j). Both losses
// are functions of the rows' l, so the gradient of a row is one coefficient times
// (one-hot(y) - softmax(z)). Per element that is two exponentials against four to
// eight bytes moved: HBM-bound.
//
// The softmax is taken about the row's maximum in fp32; a thread keeps a running
// maximum and the sum of exponentials about it, and the pairs of all threads are joined
// in a fixed order. What is formed once per row or per sequence (l, the ratio, the
// sums of l) is formed in fp64: l is a difference of numbers much larger than the
// error that a ratio near its bound may carry.
#include "row_ops.hpp"

namespace kfac {

constexpr int LT = 256;  // threads of a row's block
constexpr float LOG2E = 1.44269504088896340736f;
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

__device__ inline float exp_about(float z, float m) { return __builtin_amdgcn_exp2f((z - m) * LOG2E); }

// Maximum and sum of exp(z - maximum) of a set of logits.
struct MaxSum {
  float m, s;
};
__device__ inline MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == NEG_INF) return {m, a.s + b.s};  // nothing but -inf so far: no weight (a NaN stays in s)
  return {m, a.s * exp_about(a.m, m) + b.s * exp_about(b.m, m)};
}
template <int NT>
__device__ inline MaxSum block_join(MaxSum v, MaxSum* s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = join(v, MaxSum{__shfl_xor(v.m, o), __shfl_xor(v.s, o)});
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  MaxSum t = s[0];
  for (int i = 1; i < NT / 64; ++i) t = join(t, s[i]);
  return t;
}

// Adds n logits to a running maximum and sum.
template <int N>
__device__ inline void take(MaxSum& r, const float* z) {
  float m = r.m;
#pragma unroll
  for (int u = 0; u < N; ++u) m = fmaxf(m, z[u]);
  const float at = m == NEG_INF ? 0.f : m;
  float s = r.s * exp_about(r.m, at);
#pragma unroll
  for (int u = 0; u < N; ++u) s += exp_about(z[u], at);
  r = {m, s};
}

template <class T, int NT>
__device__ inline MaxSum row_max_sum(const KG T* z, int vocab, MaxSum* lds) {
  using C = Chunk16<T>;
  MaxSum r = {NEG_INF, 0.f};
  const int full = vocab / C::ev * C::ev;
  for (int i = threadIdx.x * C::ev; i < full; i += NT * C::ev) {
    const typename C::vec v = *reinterpret_cast<const KG typename C::vec*>(z + i);
    float x[C::ev];
#pragma unroll
    for (int u = 0; u < C::ev; ++u) x[u] = static_cast<float>(v[u]);
    take<C::ev>(r, x);
  }
  if (full + static_cast<int>(threadIdx.x) < vocab) {
    const float x = static_cast<float>(z[full + threadIdx.x]);
    take<1>(r, &x);
  }
  return block_join<NT>(r, lds);
}

// d = coef * (one-hot(y) - softmax(z)), rounded once to the row's type; each element is
// read and written by the same thread, so d may be z.
template <class T, int NT>
__device__ inline void row_gradient(const KG T* z, KG T* d, int vocab, MaxSum r, int y, float coef) {
  using C = Chunk16<T>;
  const float inv = 1.f / r.s;
  const int full = vocab / C::ev * C::ev;
  const auto one = [&](float x, int j) { return static_cast<T>(coef * ((j == y ? 1.f : 0.f) - exp_about(x, r.m) * inv)); };
  for (int i = threadIdx.x * C::ev; i < full; i += NT * C::ev) {
    const typename C::vec v = *reinterpret_cast<const KG typename C::vec*>(z + i);
    typename C::vec w;
#pragma unroll
    for (int u = 0; u < C::ev; ++u) w[u] = one(static_cast<float>(v[u]), i + u);
    *reinterpret_cast<KG typename C::vec*>(d + i) = w;
  }
  const int j = full + threadIdx.x;
  if (j < vocab) d[j] = one(static_cast<float>(z[j]), j);
}

template <class T, int NT>
__device__ inline void row_zero(KG T* d, int vocab) {
  using C = Chunk16<T>;
  const int full = vocab / C::ev * C::ev;
  typename C::vec w = {};
  for (int i = threadIdx.x * C::ev; i < full; i += NT * C::ev) *reinterpret_cast<KG typename C::vec*>(d + i) = w;
  const int j = full + threadIdx.x;
  if (j < vocab) d[j] = static_cast<T>(0.f);
}

template <int NT, class V>
__device__ inline V block_add(V v, V* s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  V t = 0;
  for (int i = 0; i < NT / 64; ++i) t += s[i];
  return t;
}

// Per sequence: how many of its rows count; per row: its sequence, -1 where it does not
// count and -2 outside every sequence.
__global__ void __launch_bounds__(LT) loss_count_kernel(LossRows a, int32_t* __restrict__ row_seq,
                                                        int32_t* __restrict__ count) {
  __shared__ int s[LT / 64];
  const int q = blockIdx.x;
  int r0, r1, n = 0;
  seq_range(a, q, q + 1, r0, r1);
  for (int t = r0 + threadIdx.x; t < r1; t += LT) {
    const bool counts = row_counts(a, t);
    row_seq[t] = counts ? q : -1;
    n += counts;
  }
  n = block_add<LT>(n, s);
  if (threadIdx.x == 0) count[q] = n;
  if (q == 0)
    for (int t = threadIdx.x; t < r0; t += LT) row_seq[t] = -2;
  if (q == a.seqs - 1)
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

template <class T>
__global__ void __launch_bounds__(LT) policy_rows_kernel(LossRows a, PolicyArgs p, const int32_t* __restrict__ row_seq,
                                                         const int32_t* __restrict__ count,
                                                         PolicyTerms* __restrict__ terms) {
  __shared__ MaxSum lds[LT / 64];
  __shared__ int lds_i[LT / 64];
  __shared__ float coef_s;
  const int t = blockIdx.x;
  int q = row_seq[t];
  if (q >= 0 && !row_counts(a, t)) q = -2;  // offsets that decrease: a row that no sequence wrote
  KG T* d = a.dlogits ? gp(static_cast<T*>(a.dlogits)) + t * a.ld_grad : nullptr;
  if (q < 0 || q >= a.seqs) {  // outside (left as it is) or not counted (no gradient)
    if (threadIdx.x == 0) {
      terms[t] = {0, 0, 0};
      if (q == -1) gp(p.logp)[t] = 0.f;
    }
    if (q == -1 && d) row_zero<T, LT>(d, a.vocab);
    return;
  }
  int n = 0;
  for (int i = threadIdx.x; i < a.seqs; i += LT) n += p.by_seq ? count[i] > 0 : count[i];
  n = block_add<LT>(n, lds_i);
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  const int y = static_cast<int>(gp(a.token)[t]);
  const double picked = static_cast<float>(z[y]);  // read before any thread may write the row
  const MaxSum r = row_max_sum<T, LT>(z, a.vocab, lds);
  if (threadIdx.x == 0) {
    const double weight = p.by_seq ? 1.0 / (static_cast<double>(n) * count[q]) : 1.0 / n;
    const double l = picked - r.m - log(static_cast<double>(r.s));
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
    gp(p.logp)[t] = static_cast<float>(l);
    terms[t] = {weight * -(over ? held : free), weight * kl, over ? weight : 0.0};
    coef_s = static_cast<float>(p.grad_scale * weight * slope);
  }
  __syncthreads();
  if (d) row_gradient<T, LT>(z, d, a.vocab, r, y, coef_s);
}

// stats: loss, its surrogate part, the mean KL, the clipped share.
__global__ void __launch_bounds__(LT) policy_finish_kernel(const PolicyTerms* __restrict__ terms, int rows,
                                                           float kl_coef, float* stats) {
  __shared__ double s[LT / 64];
  double part = 0, kl = 0, over = 0;
  for (int t = threadIdx.x; t < rows; t += LT) {
    part += terms[t].part;
    kl += terms[t].kl;
    over += terms[t].over;
  }
  part = block_add<LT>(part, s);
  kl = block_add<LT>(kl, s);
  over = block_add<LT>(over, s);
  if (threadIdx.x == 0) {
    stats[0] = static_cast<float>(kl_coef != 0.f ? part + kl_coef * kl : part);
    stats[1] = static_cast<float>(part);
    stats[2] = static_cast<float>(kl);
    stats[3] = static_cast<float>(over);
  }
}

// Softmax maximum and sum, and l, of every row that counts and lies in a sequence.
template <class T>
__global__ void __launch_bounds__(LT) pref_rows_kernel(LossRows a, MaxSum* __restrict__ row_stat,
                                                       double* __restrict__ row_logp) {
  __shared__ MaxSum lds[LT / 64];
  const int t = blockIdx.x;
  int r0, r1;
  seq_range(a, 0, a.seqs, r0, r1);
  if (t < r0 || t >= r1) return;
  if (!row_counts(a, t)) {
    if (threadIdx.x == 0) row_logp[t] = 0;
    return;
  }
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  const MaxSum r = row_max_sum<T, LT>(z, a.vocab, lds);
  if (threadIdx.x == 0) {
    row_stat[t] = r;
    row_logp[t] = static_cast<double>(static_cast<float>(z[gp(a.token)[t]])) - r.m - log(static_cast<double>(r.s));
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

// One block takes the pairs one after another: the sums of l over both sequences, the
// margin, the loss, and for each row the coefficient of its gradient.
__global__ void __launch_bounds__(LT) pref_pairs_kernel(LossRows a, PrefArgs p, const double* __restrict__ row_logp,
                                                        float* __restrict__ row_coef) {
  __shared__ double s[LT / 64];
  double loss = 0;
  for (int i = 0; i < p.pairs; ++i) {
    int r0[2], r1[2];
    double sum[2];
    for (int k = 0; k < 2; ++k) {
      const int q = i + k * p.pairs;
      seq_range(a, q, q + 1, r0[k], r1[k]);
      double v = 0;
      for (int t = r0[k] + threadIdx.x; t < r1[k]; t += LT) v += row_logp[t];
      sum[k] = block_add<LT>(v, s);
    }
    const double rc = p.ref_logp ? gp(p.ref_logp)[i] : 0.f, rr = p.ref_logp ? gp(p.ref_logp)[i + p.pairs] : 0.f;
    const double x = p.beta * ((sum[0] - rc) - (sum[1] - rr)), e = p.smooth;
    const double below = softplus(-x), above = softplus(x);  // -log sig(x), -log sig(-x)
    loss += (e != 0 ? (1 - e) * below + e * above : below) / p.pairs;
    const double slope = (e - exp(-above)) * p.beta / p.pairs;
    if (threadIdx.x == 0) {
      gp(p.margin)[i] = static_cast<float>(x);
      gp(p.seq_logp)[i] = static_cast<float>(sum[0]);
      gp(p.seq_logp)[i + p.pairs] = static_cast<float>(sum[1]);
    }
    for (int k = 0; k < 2; ++k) {
      const float c = static_cast<float>(p.grad_scale * (k ? -slope : slope));
      for (int t = r0[k] + threadIdx.x; t < r1[k]; t += LT) row_coef[t] = c;
    }
  }
  if (threadIdx.x == 0) gp(p.loss)[0] = static_cast<float>(loss);
}

template <class T>
__global__ void __launch_bounds__(LT) pref_grad_kernel(LossRows a, const MaxSum* __restrict__ row_stat,
                                                       const float* __restrict__ row_coef) {
  const int t = blockIdx.x;
  int r0, r1;
  seq_range(a, 0, a.seqs, r0, r1);
  if (t < r0 || t >= r1) return;
  KG T* d = gp(static_cast<T*>(a.dlogits)) + t * a.ld_grad;
  if (!row_counts(a, t)) {
    row_zero<T, LT>(d, a.vocab);
    return;
  }
  const KG T* z = gp(static_cast<const T*>(a.logits)) + t * a.ld;
  row_gradient<T, LT>(z, d, a.vocab, row_stat[t], static_cast<int>(gp(a.token)[t]), row_coef[t]);
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

struct PolicyWs {
  int32_t *row_seq, *count;
  PolicyTerms* terms;
  size_t bytes;
};
static PolicyWs policy_ws(void* ws, int32_t rows, int32_t seqs) {
  Carver cv(ws);
  PolicyWs w;
  w.row_seq = cv.take<int32_t>(rows);
  w.count = cv.take<int32_t>(seqs ? seqs : 1);
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
    KFAC_LAUNCH(K_LOSS_COUNT, loss_count_kernel, dim3(a.seqs), dim3(LT), 0, s, a, w.row_seq, w.count);
    KFAC_CHECK_LAUNCH("loss_count_kernel");
#define KFAC_ROWS(T)                                                                                          \
  KFAC_LAUNCH(K_POLICY_ROWS, policy_rows_kernel<T>, dim3(rows), dim3(LT), 0, s, a, p, w.row_seq, w.count, w.terms);
    KFAC_BY_TYPE(dtype, KFAC_ROWS);
#undef KFAC_ROWS
    KFAC_CHECK_LAUNCH("policy_rows_kernel");
  }
  KFAC_LAUNCH(K_POLICY_FINISH, policy_finish_kernel, dim3(1), dim3(LT), 0, s, w.terms, rows, kl_coef, stats);
  KFAC_CHECK_LAUNCH("policy_finish_kernel");
  return KFAC_OK;
}

struct PrefWs {
  MaxSum* stat;
  double* logp;
  float* coef;
  size_t bytes;
};
static PrefWs pref_ws(void* ws, int32_t rows) {
  Carver cv(ws);
  PrefWs w;
  w.stat = cv.take<MaxSum>(rows);
  w.logp = cv.take<double>(rows);
  w.coef = cv.take<float>(rows);
  w.bytes = cv.used;
  return w;
}

extern "C" kfac_status kfac_preference_loss_workspace(int32_t rows, int32_t vocab, int32_t pairs, size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  if (pairs < 0 || pairs > (1 << 23)) return fail(KFAC_ERR_INVALID, "%d pairs: out of range", pairs);
  kfac_status st = rows_validate(rows, vocab, 2 * pairs);
  if (st) return st;
  *bytes = pref_ws(nullptr, rows).bytes;
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
  const PrefWs w = pref_ws(workspace, rows);
  if ((st = check_workspace(workspace, ws_bytes, w.bytes))) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const PrefArgs p = {ref_logp, seq_logp, margin, loss, beta, label_smoothing, grad_scale, pairs};
  const bool any = rows > 0 && pairs > 0;
  if (any) {
#define KFAC_ROWS(T) KFAC_LAUNCH(K_PREF_ROWS, pref_rows_kernel<T>, dim3(rows), dim3(LT), 0, s, a, w.stat, w.logp);
    KFAC_BY_TYPE(dtype, KFAC_ROWS);
#undef KFAC_ROWS
    KFAC_CHECK_LAUNCH("pref_rows_kernel");
  }
  KFAC_LAUNCH(K_PREF_PAIRS, pref_pairs_kernel, dim3(1), dim3(LT), 0, s, a, p, w.logp, w.coef);
  KFAC_CHECK_LAUNCH("pref_pairs_kernel");
  if (any && dlogits) {
#define KFAC_ROWS(T) KFAC_LAUNCH(K_PREF_GRAD, pref_grad_kernel<T>, dim3(rows), dim3(LT), 0, s, a, w.stat, w.coef);
    KFAC_BY_TYPE(dtype, KFAC_ROWS);
#undef KFAC_ROWS
    KFAC_CHECK_LAUNCH("pref_grad_kernel");
  }
  return KFAC_OK;
}
