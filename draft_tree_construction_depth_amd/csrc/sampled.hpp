// Acceptance of drafts at a temperature, from given random numbers.
//
// Trees (drafts that are a function of the drafter's rows). At a node whose
// target row is x, with weights w(v) = exp((x_v - max x) / T) and Z their
// sum, one uniform number u places t = u Z on a line on which the node's
// children lie first, in node order, each as long as its token's weight, and
// all other tokens after them in order of id. A child hit is accepted and the
// walk goes on there; any other token hit is the round's next token. Each
// committed token then has exactly the target's distribution p = w / Z.
//
// Chains (drafts sampled from the drafter's rows q). Guess x_i stands iff
// u_i q_i(x_i) < p_i(x_i). At the first that falls the next token is drawn
// from max(0, p_i - q_i), after a whole chain from p, by the running sum in
// order of id. Committed tokens again have the target's distribution.
//
// A temperature of 0 means the first largest logit (p is its point mass).
//
// Weights, sums and comparisons are float64: a token's interval on the line
// can be as short as 1/V of it, and with V = 152 k float32 sums (1e-7 of the
// line) would move one token in fifty of a flat row. CDNA4 runs a float64
// FMA at the rate of an unpacked float32 one; exp2 is a polynomial of degree 9
// in the sums, which the vector units bound (17 instructions a logit).
//
// The row sums (records) are formed by workgroups of 256 threads, each over a
// chunk of 4 16-byte vectors per thread held in registers: its maximum, then
// the sum of its weights against that maximum. Only the rows on the path
// matter, but which they are is known only step by step: for the first depths
// the path's rows' records are formed by a launch for each depth, then those of
// all rows that the walks still going on may come to by one more (how many
// depths: accept_plan in api.hip).
//
// Measured per call, by box, rows of 152 k bf16 (parts: medians under the
// profiler, where launches take longer than in an unprofiled call). One tree of
// 64 nodes: 24 to 27 us (rows 12, finish 15: chains of dependent loads), 39 where
// the walk takes all 15 levels. 64 trees whose walks take 1.6 nodes on
// average (one in eight, greedy, 15): 120 to 128 us, six launches of 8 to 14 us
// (a full one reads 19 MB, 4 us, and has 4 us of float64 work, both behind 3 us
// of dependent loads), 47 us for the rows left, 17 us for the draw; where walks
// take 3.6 nodes 167, where every one takes all 15 levels 335 to 354, most of it
// for the rows that the last launch finds within reach. 64 chains of 16 guesses:
// 149 to 167 us, seven launches of 8 to 20 us, 21 for the rows left, 25 for
// max(0, p - q), 13 for the draw. 8 chains of 5 guesses, 32 k float32: 24 to 25 us.
#pragma once

#include "common.hpp"

namespace ddt {

constexpr int kSvThreads = 256;
constexpr int kSvVecs = 4;       // 16-byte vectors per thread and chunk
constexpr int kSvMaxS = 1025;    // chunks per row: 2^22 float32, whose first vector may start before it
constexpr int kSvMaxB = 512;     // nodes
constexpr float kSvTop = 3.402823466e38f;  // the largest finite value, which stands for +inf
constexpr int kSvChunkMax = kSvThreads * kSvVecs * 8;  // elements (bf16)
constexpr int kSvFinish = 1024;  // threads of the launches that end a walk

struct SvRec {
  double sum;  // of exp2((x - mx) / T log2 e) over the chunk
  float mx;
  int32_t arg;  // first element with x == mx (at temperature 0 only)
};

struct SvState {
  int32_t at;    // node / position of the current row
  int32_t done;  // 1: the next token comes from this row, 2: ... from max(0, p - q)
  int32_t depth;
  int32_t pad;
};

struct SvParams {
  const void* logits;  // [batch][T][V]
  const void* draft;   // chains: [batch][T-1][V]
  int64_t batch, V;
  int32_t T, L;
  const int32_t* tokens;   // [batch][T-1]
  const int32_t* parents;  // trees: [batch][T-1]
  const int32_t* count;    // nodes / kept guesses, null: T - 1
  const float* temperature;  // [batch], null: 1
  const float* u;            // [batch][L+1]
  int32_t* accepted;         // trees: [batch][L]
  int32_t* accept_len;
  int32_t* next_token;
  float* logp;  // [batch][L+1], may be null
  int32_t S;      // chunks per row
  int32_t depths;  // with a launch of their own
  int32_t slices;  // workgroups that share a request's other rows
  SvRec* rec;      // the path's rows [2][batch][S] (if depths > 0), all rows [batch][T][S]
  SvRec* rec_q;    // chains: the same of the drafter's rows (T-1 of them)
  SvState* state;  // [L+2][batch], after each launch
  double* rest;    // chains: [batch][S] sums of max(0, p - q)
};

typedef unsigned int sv_u32x4 __attribute__((ext_vector_type(4)));

template <int DT>
struct SvVec {
  static constexpr int N = DT == 0 ? 8 : 4;  // elements of a 16-byte vector
  sv_u32x4 r;
  // element e; NaN counts as -inf, +inf as the largest finite value
  __device__ __forceinline__ float raw(int e) const {
    return DT == 0 ? __uint_as_float(e & 1 ? r[e >> 1] & 0xFFFF0000u : r[e >> 1] << 16)
                   : __uint_as_float(r[e & 3]);
  }
  __device__ __forceinline__ float at(int e) const {
    const float x = raw(e);
    return x == x ? fminf(x, kSvTop) : -INFINITY;
  }
};

// Elements [e0, e0 + N) of the row that starts at element r0; -inf outside it.
template <int DT>
__device__ __forceinline__ SvVec<DT> sv_load(const void* base, int64_t r0, int64_t e0, int64_t V) {
  constexpr int N = SvVec<DT>::N;
  SvVec<DT> x;
  if (e0 >= 0 && e0 + N <= V && ((r0 + e0) & (N - 1)) == 0) {
    x.r = DT == 0 ? *(const sv_u32x4*)((const uint16_t*)base + r0 + e0)
                  : *(const sv_u32x4*)((const float*)base + r0 + e0);
  } else if (DT == 0) {
    const uint16_t* p = (const uint16_t*)base + r0;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const uint32_t lo = e0 + e >= 0 && e0 + e < V ? p[e0 + e] : 0xFF80u;
      const uint32_t hi = e0 + e + 1 >= 0 && e0 + e + 1 < V ? p[e0 + e + 1] : 0xFF80u;
      x.r[e >> 1] = lo | hi << 16;
    }
  } else {
    const uint32_t* p = (const uint32_t*)base + r0;
#pragma unroll
    for (int e = 0; e < 4; ++e) x.r[e] = e0 + e >= 0 && e0 + e < V ? p[e0 + e] : 0xFF800000u;
  }
  return x;
}

template <int DT>
__device__ __forceinline__ float sv_logit(const void* base, int64_t r0, int64_t e) {
  SvVec<DT> x;
  x.r[0] = DT == 0 ? (uint32_t)((const uint16_t*)base)[r0 + e] : ((const uint32_t*)base)[r0 + e];
  return x.at(0);
}

// 2^y for y <= 0 (anything below -1100, and NaN, gives 0): 2^k times the
// Taylor polynomial of exp on [-ln2/2, ln2/2], within 9e-15 of the result.
__device__ __forceinline__ double sv_exp2(double y) {
  y = fmax(y, -1100.0);
  const double k = rint(y);
  const double z = (y - k) * 0.6931471805599453094;
  double s = 1.0 / 39916800.0;
  s = fma(s, z, 1.0 / 3628800.0);
  s = fma(s, z, 1.0 / 362880.0);
  s = fma(s, z, 1.0 / 40320.0);
  s = fma(s, z, 1.0 / 5040.0);
  s = fma(s, z, 1.0 / 720.0);
  s = fma(s, z, 1.0 / 120.0);
  s = fma(s, z, 1.0 / 24.0);
  s = fma(s, z, 1.0 / 6.0);
  s = fma(s, z, 0.5);
  s = fma(s, z, 1.0);
  s = fma(s, z, 1.0);
  return ldexp(s, (int)k);
}

// The same for the sums: y within [-1000, 0] (what is below counts as 2^-1000),
// 2^f by the polynomial through its values at the ten Chebyshev nodes of
// [-1/2, 1/2], its constant 1.0000000000000135 set to 1 (within 3.8e-14 of
// the result), 2^k added to the exponent's bits.
__device__ __forceinline__ double sv_exp2_fast(double y) {
  y = fmax(y, -1000.0);
  const double big = 6755399441055744.0;  // 1.5 * 2^52: the sum's low bits are k
  const double t = y + big;
  const double f = y - (t - big);
  double s = 1.0205905413765595471e-07;
  s = fma(s, f, 1.3259645244887110601e-06);
  s = fma(s, f, 1.5252672924850737155e-05);
  s = fma(s, f, 0.00015403433751251009655);
  s = fma(s, f, 0.0013333558200794592453);
  s = fma(s, f, 0.0096181291939343126207);
  s = fma(s, f, 0.055504108664651670424);
  s = fma(s, f, 0.24022650695640340723);
  s = fma(s, f, 0.69314718055994617441);
  s = fma(s, f, 1.0);
  const uint64_t k = (uint64_t)__builtin_bit_cast(uint64_t, t) << 52;
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, s) + k);
}

// Inclusive scan of one double per lane over the wave (every lane active), by
// DPP as in wave_incl_scan.
template <int CTRL, int ROWS>
__device__ __forceinline__ double sv_shifted(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_incl_scan_f64(double x) {
  x += sv_shifted<0x111, 0xf>(x);
  x += sv_shifted<0x112, 0xf>(x);
  x += sv_shifted<0x114, 0xf>(x);
  x += sv_shifted<0x118, 0xf>(x);
  x += sv_shifted<0x142, 0xa>(x);
  x += sv_shifted<0x143, 0xc>(x);
  return x;
}

struct SvHeat {
  double s;  // log2(e) / temperature
  bool greedy;
};

__device__ __forceinline__ SvHeat sv_heat(const SvParams& p, int64_t b) {
  const float t = p.temperature ? p.temperature[b] : 1.0f;
  SvHeat h;
  h.greedy = !(t > 0.0f);
  h.s = h.greedy ? 0.0 : 1.4426950408889634074 / (double)t;
  return h;
}

__device__ __forceinline__ double sv_uniform(const SvParams& p, int64_t b, int i) {
  const float u = p.u[b * (p.L + 1) + i];
  return u >= 0.0f ? (u < 1.0f ? (double)u : 1.0 - 0x1p-24) : 0.0;
}

__device__ __forceinline__ int sv_count(const SvParams& p, int64_t b) {
  const int n = p.count ? p.count[b] : p.T - 1;
  return n < 0 ? 0 : (n > p.T - 1 ? p.T - 1 : n);
}

// A row's distribution: weights exp2((x - M) s), their sum Z; greedy: the
// point mass at arg.
struct SvRow {
  double M, Z, s;
  int arg;
  bool greedy;
  __device__ __forceinline__ double weight(float x, int64_t id) const {
    if (greedy) return id == arg ? 1.0 : 0.0;
    return sv_exp2(((double)x - M) * s);
  }
};

// Lanes that combine one row's records: 16, 32 or 64.
__device__ __forceinline__ int sv_lanes(int S) { return S <= 16 ? 16 : (S <= 32 ? 32 : 64); }

// Combines a row's S records by groups of `lanes` lanes, a row each.
__device__ __forceinline__ SvRow sv_combine(const SvRec* rec, int S, const SvHeat& h, int lanes) {
  const int l = threadIdx.x & (lanes - 1);
  float m = -INFINITY;
  SvRec r{0.0, -INFINITY, 0x7FFFFFFF};
  if (l < S) r = rec[l];
  m = r.mx;
  for (int c = l + lanes; c < S; c += lanes) m = fmaxf(m, rec[c].mx);
  for (int d = 1; d < lanes; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const bool any = m > -INFINITY;
  double z = any ? r.sum * sv_exp2(((double)r.mx - (double)m) * h.s) : 0.0;
  int arg = r.mx == m ? r.arg : 0x7FFFFFFF;
  for (int c = l + lanes; c < S; c += lanes) {
    r = rec[c];
    if (any) z += r.sum * sv_exp2(((double)r.mx - (double)m) * h.s);
    if (r.mx == m && r.arg < arg) arg = r.arg;
  }
  for (int d = 1; d < lanes; d <<= 1) {
    z += __shfl_xor(z, d);
    const int o = __shfl_xor(arg, d);
    arg = o < arg ? o : arg;
  }
  SvRow row;
  row.M = (double)m;
  row.s = h.s;
  row.greedy = h.greedy;
  row.Z = !any ? 0.0 : (h.greedy ? 1.0 : z);
  row.arg = any && h.greedy ? arg : -1;
  return row;
}

// The same by every wave for itself.
__device__ __forceinline__ SvRow sv_combine(const SvRec* rec, int S, const SvHeat& h) {
  return sv_combine(rec, S, h, sv_lanes(S));
}

// This thread's part of a chunk's sum of weights against its maximum m.
template <int DT>
__device__ __forceinline__ double sv_sum(const SvVec<DT> (&x)[kSvVecs], float m, const SvHeat& h) {
  constexpr int N = SvVec<DT>::N;
  const double ms = (double)m * h.s;
  double z[2] = {0.0, 0.0};
  if (fabs(ms) < 1024.0 && m < kSvTop) {
    // (x - m) s as x s - m s is within 2^-43 then; NaN and -inf end at the
    // least weight by the maximum in sv_exp2_fast, and there is no +inf
#pragma unroll
    for (int i = 0; i < kSvVecs; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) z[e & 1] += sv_exp2_fast(fma((double)x[i].raw(e), h.s, -ms));
  } else {
#pragma unroll
    for (int i = 0; i < kSvVecs; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) z[e & 1] += sv_exp2(((double)x[i].at(e) - (double)m) * h.s);
  }
  return z[0] + z[1];
}

// One chunk's record.
template <int DT>
__device__ __forceinline__ void sv_chunk(const void* base, int64_t r0, int64_t V, int c,
                                         const SvHeat& h, SvRec* out) {
  constexpr int N = SvVec<DT>::N, NW = kSvThreads / kWave;
  __shared__ float s_m[NW];
  __shared__ double s_s[NW];
  __shared__ int s_a[NW];
  const int tid = threadIdx.x, w = tid >> 6;
  const int64_t v0 = (int64_t)c * kSvThreads * kSvVecs;
  const int off = (int)(r0 & (N - 1));  // vectors are aligned in memory, not to the row
  SvVec<DT> x[kSvVecs];
#pragma unroll
  for (int i = 0; i < kSvVecs; ++i)
    x[i] = sv_load<DT>(base, r0, (v0 + i * kSvThreads + tid) * N - off, V);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSvVecs; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, x[i].raw(e));  // (passes NaN over)
  m = wave_max(fminf(m, kSvTop));
  if ((tid & 63) == 0) s_m[w] = m;
  __syncthreads();
  m = s_m[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) m = fmaxf(m, s_m[i]);
  if (h.greedy) {
    int arg = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kSvVecs; ++i)
#pragma unroll
      for (int e = N - 1; e >= 0; --e)
        if (x[i].at(e) == m) {
          const int id = (int)((v0 + i * kSvThreads + tid) * N - off) + e;
          arg = id < arg && id >= 0 ? id : arg;
        }
    arg = wave_min(arg);
    if ((tid & 63) == 0) s_a[w] = arg;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < NW; ++i) arg = s_a[i] < arg ? s_a[i] : arg;
      *out = SvRec{0.0, m, arg};
    }
  } else {
    const double z = wave_sum(sv_sum<DT>(x, m, h));
    if ((tid & 63) == 0) s_s[w] = z;
    __syncthreads();
    if (tid == 0) {
      double all = z;
      for (int i = 1; i < NW; ++i) all += s_s[i];
      *out = SvRec{m > -INFINITY ? all : 0.0, m, 0x7FFFFFFF};
    }
  }
}

__device__ __forceinline__ float sv_logp(double w, double Z) {
  return Z > 0.0 ? (float)(log(w) - log(Z)) : -INFINITY;
}

// Where the records of a row lie: by request and the parity of the depth for
// the first depths, by row for the others.
__device__ __forceinline__ int64_t sv_rec_at(const SvParams& p, int64_t b, int at, int d, int per) {
  if (d < p.depths) return ((int64_t)(d & 1) * p.batch + b) * p.S;
  return ((p.depths > 0 ? 2 * p.batch : 0) + b * per + at) * p.S;
}

// ---- trees: the line at a node ------------------------------------------------
// A node's key: its parent and its token in one word (B <= 512, V <= 2^22); a
// node that cannot be accepted has none.
constexpr uint32_t kSvNoKey = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t sv_key(const SvParams& p, int64_t b, int j) {
  if (j >= p.T - 1) return kSvNoKey;
  const int par = p.parents[b * (p.T - 1) + j], tok = p.tokens[b * (p.T - 1) + j];
  if (par < 0 || par > j || tok < 0 || tok >= p.V) return kSvNoKey;
  return (uint32_t)par << 22 | (uint32_t)tok;
}

// Walk state of a request's tree in LDS, by node j (number j + 1).
struct SvTree {
  uint32_t key[kSvMaxB];
  double w[kSvMaxB];  // weight of the node's token in its parent's row
  // the decision: child hit (-1: none), all children's weight, and the
  // children that take a part of the line: their tokens and weights
  int pick, kids;
  double edge;
  int tok[kSvMaxB];
  double part[kSvMaxB];
};

// Where position `at` of the line falls at a node, by one wave: t.pick,
// t.edge and, for the draw after it, the children's parts. A token that an
// earlier sibling carries already takes no second part.
__device__ __forceinline__ void sv_hit(SvTree& t, int node, int n, double at) {
  const int lane = threadIdx.x & 63;
  double base = 0.0;
  int pick = -1, kept = 0;
  for (int j0 = 0; j0 < n; j0 += kWave) {
    const int j = j0 + lane;
    const uint32_t key = j < n ? t.key[j] : kSvNoKey;
    bool kid = key != kSvNoKey && (int)(key >> 22) == node;
    uint64_t kids = __ballot(kid);
    if (!kids) continue;
    const int tok = (int)(key & 0x3FFFFFu);
    for (int i = 0; i < kept; ++i) kid = kid && t.tok[i] != tok;
    for (uint64_t left = kids; left & (left - 1); left &= left - 1) {
      const int l = __builtin_ctzll(left);
      kid = kid && (lane <= l || tok != __builtin_amdgcn_readlane(tok, l));
    }
    kids = __ballot(kid);
    const double w = kid ? t.w[j] : 0.0;
    const double cum = base + wave_incl_scan_f64(w);
    // (the scan's rounding may pass `at` at a child without weight)
    const uint64_t hit = __ballot(kid && w > 0.0 && at < cum);
    if (kid) {
      t.tok[kept + lanes_below(kids)] = tok;
      t.part[kept + lanes_below(kids)] = w;
    }
    kept += __popcll(kids);
    base = lane_value(cum, 63);
    if (hit) {
      pick = j0 + __builtin_ctzll(hit);
      break;
    }
  }
  if (lane == 0) {
    t.pick = pick;
    t.edge = base;
    t.kids = kept;
  }
}

// The walk's state after `step` decisions, the last of them made here from
// the records of the launch before; every workgroup of a request makes the same
// one, and the one for which `first` is set writes it down.
template <int DT>
__device__ __forceinline__ SvState sv_decide(const SvParams& p, int64_t b, int step,
                                             const SvHeat& h, SvState st, bool first, SvTree& sh) {
  if (!st.done) {
    const int tid = threadIdx.x, d = step - 1;
    const uint32_t k0 = sv_key(p, b, tid), k1 = sv_key(p, b, tid + kSvThreads);
    const int n = d < p.L ? sv_count(p, b) : 0;
    // the node's children
    const int64_t r0 = (b * p.T + st.at) * p.V;
    const bool kid0 = k0 != kSvNoKey && (int)(k0 >> 22) == st.at;
    const bool kid1 = k1 != kSvNoKey && (int)(k1 >> 22) == st.at;
    const int t0 = (int)(k0 & 0x3FFFFFu), t1 = (int)(k1 & 0x3FFFFFu);
    const float x0 = kid0 ? sv_logit<DT>(p.logits, r0, t0) : 0.0f;
    const float x1 = kid1 ? sv_logit<DT>(p.logits, r0, t1) : 0.0f;
    const SvRow row = sv_combine(p.rec + sv_rec_at(p, b, st.at, d, p.T), p.S, h);
    sh.key[tid] = kid0 ? k0 : kSvNoKey;
    sh.key[tid + kSvThreads] = kid1 ? k1 : kSvNoKey;
    sh.w[tid] = kid0 ? row.weight(x0, t0) : 0.0;
    sh.w[tid + kSvThreads] = kid1 ? row.weight(x1, t1) : 0.0;
    __syncthreads();
    if (tid < kWave) sv_hit(sh, st.at, n, sv_uniform(p, b, d) * row.Z);
    __syncthreads();
    if (sh.pick >= 0) {
      if (first && tid == 0) {
        p.accepted[b * p.L + d] = sh.pick + 1;
        if (p.logp) p.logp[b * (p.L + 1) + d] = sv_logp(sh.w[sh.pick], row.Z);
      }
      st.at = sh.pick + 1;
      st.depth = step;
    } else {
      st.done = 1;
    }
  }
  if (first && threadIdx.x == 0) p.state[(int64_t)step * p.batch + b] = st;
  return st;
}

// One step of the walk for every request, then one chunk of the next row's
// records.
template <int DT>
__global__ __launch_bounds__(kSvThreads) void sv_step_kernel(SvParams p, int step) {
  __shared__ SvTree sh;
  const int64_t b = blockIdx.x / p.S;
  const int c = (int)(blockIdx.x - b * p.S);
  const SvHeat h = sv_heat(p, b);
  SvState st{0, 0, 0, 0};
  if (step > 0)
    st = sv_decide<DT>(p, b, step, h, p.state[(int64_t)(step - 1) * p.batch + b], c == 0, sh);
  else if (c == 0 && threadIdx.x == 0)
    p.state[b] = st;
  if (st.done) return;
  sv_chunk<DT>(p.logits, (b * p.T + st.at) * p.V, p.V, c, h,
               p.rec + sv_rec_at(p, b, st.at, step, p.T) + c);
}

// Whether row r is node `node` or below it (parents come before their children).
__device__ __forceinline__ bool sv_below(const int32_t* parent, int r, int node) {
  while (r > node) r = parent[r - 1];
  return r == node;
}

// The last step, then one chunk of the records of every row that the walk may
// still come to: the node's and those below it, dealt to the request's
// workgroups of this chunk in turn.
template <int DT>
__global__ __launch_bounds__(kSvThreads) void sv_rows_kernel(SvParams p) {
  __shared__ SvTree sh;
  __shared__ int32_t s_parent[kSvMaxB];
  const int64_t id = blockIdx.x / p.S, b = id / p.slices;
  const int c = (int)(blockIdx.x - id * p.S), slice = (int)(id - b * p.slices);
  const bool first = c == 0 && slice == 0;
  const SvHeat h = sv_heat(p, b);
  const int n = sv_count(p, b);
  SvState st{0, 0, 0, 0};
  if (p.depths > 0) {
    st = p.state[(int64_t)(p.depths - 1) * p.batch + b];
    if (!st.done) {
      for (int j = threadIdx.x; j < p.T - 1; j += kSvThreads) {
        const int par = p.parents[b * (p.T - 1) + j];
        s_parent[j] = par > j ? -1 : par;
      }
    }
    st = sv_decide<DT>(p, b, p.depths, h, st, first, sh);
    if (st.done) return;
  }
  const int last = st.depth < p.L ? n : st.at;
  for (int r = st.at + slice; r <= last; r += p.slices) {  // uniform
    if (p.depths > 0 && !sv_below(s_parent, r, st.at)) continue;
    __syncthreads();  // the row before is done with sv_chunk's LDS
    const int64_t row = b * p.T + r;
    sv_chunk<DT>(p.logits, row * p.V, p.V, c, h,
                 p.rec + sv_rec_at(p, b, r, p.depths, p.T) + c);
  }
}

// ---- the draw of the next token --------------------------------------------------
template <int NT>
struct SvDraw {
  static constexpr int VECS = kSvThreads * kSvVecs / NT;  // vectors per thread
  double z;
  int found, last;
  double seg[VECS][NT / kWave];
  uint32_t bits[kSvChunkMax / 32];
  double rest[kSvMaxS];
};

// Draws from the weights of a chunk (minus q's for PQ, without the tokens
// marked in sh.bits): the first element whose running sum passes t, else the
// last with any weight, else -1. Every thread calls it.
template <int DT, bool PQ, int NT>
__device__ int sv_draw_chunk(const SvParams& p, int64_t rp, int64_t rq, int c, const SvRow& row,
                             const SvRow& rowq, bool marked, double t, SvDraw<NT>& sh) {
  constexpr int N = SvVec<DT>::N, NW = NT / kWave, VECS = SvDraw<NT>::VECS;
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int64_t v0 = (int64_t)c * kSvThreads * kSvVecs;
  const int off = (int)(rp & (N - 1));
  const double zp = 1.0 / row.Z, zq = PQ ? 1.0 / rowq.Z : 0.0;
  SvVec<DT> x[VECS], y[PQ ? VECS : 1];
  double incl[VECS];
  uint32_t some = 0;  // vectors with any weight
  auto weight = [&](int i, int e) -> double {
    const int64_t id = (v0 + i * NT + tid) * N - off + e;
    if (id < 0 || id >= p.V) return 0.0;
    double a = row.weight(x[i].at(e), id);
    if (PQ) a = fmax(a * zp - rowq.weight(y[PQ ? i : 0].at(e), id) * zq, 0.0);
    const int k = (int)(id + off - v0 * N);
    if (marked && (sh.bits[k >> 5] >> (k & 31)) & 1) a = 0.0;
    return a;
  };
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int64_t e0 = (v0 + i * NT + tid) * N - off;
    x[i] = sv_load<DT>(p.logits, rp, e0, p.V);
    if (PQ) y[PQ ? i : 0] = sv_load<DT>(p.draft, rq, e0, p.V);
  }
  if (tid == 0) sh.found = sh.last = -1;
  int last = -1;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const double a = weight(i, e);
      sum += a;
      if (a > 0.0) last = i * N + e;
    }
    incl[i] = wave_incl_scan_f64(sum);
    some |= (sum > 0.0 ? 1u : 0u) << i;
    if (lane == 63) sh.seg[i][w] = incl[i];
  }
  __syncthreads();
  double run = 0.0;
  int hit = -1;
  for (int g = 0; g < VECS * NW; ++g) {
    const double s = sh.seg[g / NW][g % NW];
    if (run + s > t) {
      hit = g;
      break;
    }
    run += s;
  }
  if (hit >= 0) {
    if (w == hit % NW) {
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        if (i != hit / NW) continue;
        // the scan's rounding may pass t at a vector without weight: the next
        // one that has any, or the last
        const uint64_t any = __ballot(some >> i & 1), over = __ballot(run + incl[i] > t) & any;
        const int l = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(any);
        const double before = __shfl_up(incl[i], 1);
        if (lane == l) {
          double cum = run + (lane > 0 ? before : 0.0);
          int at = -1;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const double a = weight(i, e);
            const bool open = at < 0 || !(cum > t);
            cum += a;
            if (a > 0.0 && open) at = e;
          }
          sh.found = (int)((v0 + i * NT + tid) * N - off) + at;
        }
      }
    }
  } else {
    // the last element with any weight
    const int id =
        last < 0 ? -1 : (int)((v0 + (last / N) * NT + tid) * N - off) + last % N;
    const int top = wave_max(id);
    if (lane == 0) atomicMax(&sh.found, top);
  }
  __syncthreads();
  const int found = sh.found;
  __syncthreads();
  return found;
}

// Draws the next token from a row whose chunk sums are sh.rest[0 .. S): the
// chunk that t falls into, then the element; where rounding leaves no weight
// there, the chunks behind it, then those before it. tok: the n_marked tokens
// without a part. Every thread calls it.
template <int DT, bool PQ, int NT>
__device__ int sv_draw(const SvParams& p, int64_t rp, int64_t rq, const SvRow& row,
                       const SvRow& rowq, const int* tok, int n_marked, double t,
                       SvDraw<NT>& sh) {
  constexpr int N = SvVec<DT>::N;
  const int tid = threadIdx.x;
  double before = 0.0;
  int c0 = -1;
  for (int c = 0; c < p.S; ++c) {
    if (before + sh.rest[c] > t) {
      c0 = c;
      break;
    }
    before += sh.rest[c];
  }
  const bool past_end = c0 < 0;
  if (past_end) c0 = p.S - 1;
  const int off = (int)(rp & (N - 1));
  for (int a = 0; a < p.S; ++a) {
    const int c = c0 + a < p.S ? c0 + a : p.S - 1 - a;
    // behind c0 the first weight is taken, before it (or past the end) the last
    const double tc = a == 0 && !past_end ? fmax(t - before, 0.0) : (c > c0 ? 0.0 : 1e300);
    if (n_marked > 0) {
      for (int i = tid; i < kSvChunkMax / 32; i += NT) sh.bits[i] = 0;
      __syncthreads();
      for (int i = tid; i < n_marked; i += NT) {
        const int64_t k = (int64_t)tok[i] + off - (int64_t)c * kSvThreads * kSvVecs * N;
        if (k >= 0 && k < kSvThreads * kSvVecs * N) atomicOr(&sh.bits[k >> 5], 1u << (k & 31));
      }
      __syncthreads();
    }
    const int id = sv_draw_chunk<DT, PQ, NT>(p, rp, rq, c, row, rowq, n_marked > 0, tc, sh);
    if (id >= 0) return id;
  }
  return -1;
}

template <bool CHAIN>
__device__ void sv_tail(const SvParams& p, int64_t b, int depth, int token, double w, double Z) {
  for (int i = depth + threadIdx.x; i <= p.L; i += blockDim.x) {
    if (!CHAIN && i < p.L) p.accepted[b * p.L + i] = -1;
    if (p.logp)
      p.logp[b * (p.L + 1) + i] = i > depth ? 0.0f : (token < 0 ? -INFINITY : sv_logp(w, Z));
  }
  if (threadIdx.x == 0) {
    p.accept_len[b] = depth;
    p.next_token[b] = token;
  }
}

// Trees: the rest of the walk and the next token, one workgroup per request. Every row's sums and every node's weight are formed
// side by side first, so that the walk itself only reads LDS.
template <int DT>
__global__ __launch_bounds__(kSvFinish) void sv_finish_kernel(SvParams p) {
  constexpr int NT = kSvFinish, N = SvVec<DT>::N;
  __shared__ SvTree sh;
  __shared__ SvDraw<NT> dr;
  __shared__ double s_Z[kSvMaxB + 1];
  __shared__ float s_M[kSvMaxB + 1];
  __shared__ int s_arg[kSvMaxB + 1];
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x;
  const SvHeat h = sv_heat(p, b);
  uint32_t key = sv_key(p, b, tid);
  const int count = sv_count(p, b);
  if (tid >= count) key = kSvNoKey;
  int node = 0, d = 0;
  bool ended = false;
  if (p.depths > 0) {
    const SvState st = p.state[(int64_t)p.depths * p.batch + b];
    node = st.at;
    d = st.depth;
    // the walk has ended here; its node's line is formed again
    ended = st.done != 0;
    if (key != kSvNoKey && (ended ? (int)(key >> 22) != node : (int)(key >> 22) < node)) key = kSvNoKey;
  }
  const int par = (int)(key >> 22), tok = (int)(key & 0x3FFFFFu);
  const float x = key != kSvNoKey ? sv_logit<DT>(p.logits, (b * p.T + par) * p.V, tok) : 0.0f;
  if (tid < kSvMaxB) sh.key[tid] = key;
  // the rows' maxima and sums: a group of lanes takes a row (a walk that has
  // ended: the node's only; of the others those not below the node are old
  // records, which no decision reads)
  const int lanes = sv_lanes(p.S), end = ended || node > count ? node : count;
  for (int r0 = node; r0 <= end; r0 += NT / lanes) {  // uniform
    const int r = r0 + tid / lanes;
    const SvRow row =
        sv_combine(p.rec + sv_rec_at(p, b, r <= end ? r : end, d, p.T), p.S, h, lanes);
    if (r <= end && (tid & (lanes - 1)) == 0) {
      s_Z[r] = row.Z;
      s_M[r] = (float)row.M;
      s_arg[r] = row.arg;
    }
  }
  __syncthreads();
  auto row_of = [&](int r) {
    SvRow row;
    row.M = (double)s_M[r];
    row.Z = s_Z[r];
    row.s = h.s;
    row.arg = s_arg[r];
    row.greedy = h.greedy;
    return row;
  };
  if (tid < kSvMaxB) sh.w[tid] = key != kSvNoKey ? row_of(par).weight(x, tok) : 0.0;
  __syncthreads();
  if (tid < kWave) {
    for (;;) {
      sv_hit(sh, node, d < p.L ? count : 0, ended ? 1e300 : sv_uniform(p, b, d) * s_Z[node]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int pick = sh.pick;
      if (pick < 0) break;
      if (tid == 0) {
        p.accepted[b * p.L + d] = pick + 1;
        if (p.logp) p.logp[b * (p.L + 1) + d] = sv_logp(sh.w[pick], s_Z[node]);
      }
      node = pick + 1;
      ++d;
    }
    if (tid == 0) {
      dr.found = node;
      dr.last = d;
    }
  }
  __syncthreads();
  node = dr.found;
  d = dr.last;
  const SvRow row = row_of(node);
  const int n = sh.kids;
  int token = -1;
  double w = 0.0;
  if (row.Z > 0.0 && row.greedy) {
    token = row.arg;
    w = 1.0;
  } else if (row.Z > 0.0) {
    // the chunks' weights without the children's
    const SvRec* rec = p.rec + sv_rec_at(p, b, node, d, p.T);
    const int64_t r0 = (b * p.T + node) * p.V;
    const int off = (int)(r0 & (N - 1));
    const double at = sv_uniform(p, b, d) * row.Z - sh.edge;
    for (int c = tid; c < p.S; c += NT) {
      double s = rec[c].sum * sv_exp2(((double)rec[c].mx - row.M) * row.s);
      for (int j = 0; j < n; ++j)
        if ((sh.tok[j] + off) / (kSvThreads * kSvVecs * N) == c) s -= sh.part[j];
      dr.rest[c] = fmax(s, 0.0);
    }
    __syncthreads();
    token = sv_draw<DT, false, NT>(p, r0, 0, row, row, sh.tok, n, at, dr);
    if (token >= 0) w = row.weight(sv_logit<DT>(p.logits, r0, token), token);
  }
  sv_tail<false>(p, b, d, token, w, row.Z);
}

// ---- chains ----------------------------------------------------------------------
// The tests of guesses, a pair of lane groups each: even groups combine the
// target's row, odd ones the drafter's, and both form the test. i: this pair's
// guess (an existing one).
template <int DT>
__device__ bool sv_test(const SvParams& p, int64_t b, int i, const SvHeat& h, int lanes, double& wt,
                        SvRow& row) {
  const int P = p.T - 1;
  const bool q = (threadIdx.x / lanes) & 1;
  const int token = p.tokens[b * P + i];
  const bool in = token >= 0 && token < p.V;
  const float x = !in ? 0.0f
                  : q ? sv_logit<DT>(p.draft, (b * P + i) * p.V, token)
                      : sv_logit<DT>(p.logits, (b * p.T + i) * p.V, token);
  const SvRow mine = sv_combine(q ? p.rec_q + sv_rec_at(p, b, i, i, P)
                                  : p.rec + sv_rec_at(p, b, i, i, p.T),
                                p.S, h, lanes);
  const double w = in ? mine.weight(x, token) : 0.0;
  const double wo = __shfl_xor(w, lanes), Zo = __shfl_xor(mine.Z, lanes);
  const double wp = q ? wo : w, wq = q ? w : wo, Zp = q ? Zo : mine.Z, Zq = q ? mine.Z : Zo;
  wt = wp;
  row = mine;
  row.Z = Zp;
  // (a drafter's row with every token masked has q = 0)
  return in && sv_uniform(p, b, i) * wq * Zp < wp * (Zq > 0.0 ? Zq : 1.0);
}

// As sv_decide: the state after the test of guess step - 1.
template <int DT>
__device__ __forceinline__ SvState sv_chain_decide(const SvParams& p, int64_t b, int step,
                                                   const SvHeat& h, SvState st, int keep,
                                                   bool first) {
  const int pair = p.S <= 16 ? 16 : 32;  // two groups to a wave at least
  if (!st.done) {
    double wt = 0.0;
    SvRow row;
    if (st.at >= keep) {
      st.done = 1;
    } else if (sv_test<DT>(p, b, st.at, h, pair, wt, row)) {  // every pair the same
      if (first && threadIdx.x == 0 && p.logp) p.logp[b * (p.L + 1) + st.at] = sv_logp(wt, row.Z);
      st.at = st.depth = step;
    } else {
      st.done = 2;
    }
  }
  if (first && threadIdx.x == 0) p.state[(int64_t)step * p.batch + b] = st;
  return st;
}

// One step of a chain for every request, then one chunk of the next rows'
// records.
template <int DT>
__global__ __launch_bounds__(kSvThreads) void sv_chain_step_kernel(SvParams p, int step) {
  const int64_t b = blockIdx.x / (2 * p.S);
  int c = (int)(blockIdx.x - b * 2 * p.S);
  const bool q = c >= p.S, first = c == 0;
  if (q) c -= p.S;
  const SvHeat h = sv_heat(p, b);
  const int keep = sv_count(p, b);
  SvState st{0, 0, 0, 0};
  if (step > 0)
    st = sv_chain_decide<DT>(p, b, step, h, p.state[(int64_t)(step - 1) * p.batch + b], keep,
                             first);
  else if (first && threadIdx.x == 0)
    p.state[b] = st;
  if (st.done || (q && st.at >= keep)) return;
  const int per = q ? p.T - 1 : p.T;
  sv_chunk<DT>(q ? p.draft : p.logits, (b * per + st.at) * p.V, p.V, c, h,
               (q ? p.rec_q : p.rec) + sv_rec_at(p, b, st.at, step, per) + c);
}

// The last step, then one chunk of the records of all rows left.
template <int DT>
__global__ __launch_bounds__(kSvThreads) void sv_chain_rows_kernel(SvParams p) {
  const int64_t id = blockIdx.x / p.S, b = id / p.slices;
  const int c = (int)(blockIdx.x - id * p.S), slice = (int)(id - b * p.slices);
  const SvHeat h = sv_heat(p, b);
  const int keep = sv_count(p, b);
  SvState st{0, 0, 0, 0};
  if (p.depths > 0) {
    st = sv_chain_decide<DT>(p, b, p.depths, h, p.state[(int64_t)(p.depths - 1) * p.batch + b],
                             keep, c == 0 && slice == 0);
    if (st.done) return;
  }
  for (int j = slice; j <= 2 * (keep - st.at); j += p.slices) {  // uniform
    const bool q = j & 1;
    const int i = st.at + (j >> 1), per = q ? p.T - 1 : p.T;
    __syncthreads();  // the row before is done with sv_chunk's LDS
    sv_chunk<DT>(q ? p.draft : p.logits, (b * per + i) * p.V, p.V, c, h,
                 (q ? p.rec_q : p.rec) + sv_rec_at(p, b, i, p.depths, per) + c);
  }
}

// Chains: the tests that are left, all of them side by side, and chunk sums of max(0, p - q) where a guess fell. Every workgroup of a request
// forms the same state.
constexpr int kSvRest = 512;

template <int DT>
__global__ __launch_bounds__(kSvRest) void sv_chain_rest_kernel(SvParams p) {
  constexpr int N = SvVec<DT>::N, NW = kSvRest / kWave, VECS = kSvThreads * kSvVecs / kSvRest;
  __shared__ double s_s[NW];
  __shared__ float s_logp[DDT_MAX_L];
  __shared__ int s_ok[DDT_MAX_L];
  const int64_t b = blockIdx.x / p.S;
  const int c = (int)(blockIdx.x - b * p.S), tid = threadIdx.x, wave = tid >> 6;
  const SvHeat h = sv_heat(p, b);
  const int keep = sv_count(p, b);
  SvState st{0, 0, 0, 0};
  if (p.depths > 0) st = p.state[(int64_t)p.depths * p.batch + b];
  if (!st.done) {
    const int lanes = p.S <= 16 ? 16 : 32, pairs = kSvRest / (2 * lanes);
    const int g = tid / (2 * lanes);
    const int i0 = st.at;
    for (int j = i0; j < keep; j += pairs) {  // uniform
      const int i = j + g < keep ? j + g : keep - 1;
      double wt = 0.0;
      SvRow row;
      const bool ok = sv_test<DT>(p, b, i, h, lanes, wt, row);
      if ((tid & (2 * lanes - 1)) == 0 && j + g < keep) {
        s_ok[i] = ok;
        s_logp[i] = sv_logp(wt, row.Z);
      }
    }
    __syncthreads();
    int at = i0;
    while (at < keep && s_ok[at]) ++at;
    if (c == 0 && p.logp)
      for (int i = i0 + tid; i < at; i += kSvRest) p.logp[b * (p.L + 1) + i] = s_logp[i];
    st.at = st.depth = at;
    st.done = at < keep ? 2 : 1;
  }
  if (c == 0 && tid == 0) p.state[(int64_t)(p.L + 1) * p.batch + b] = st;
  if (st.done != 2 || h.greedy) return;
  const int64_t rp = (b * p.T + st.at) * p.V, rq = (b * (p.T - 1) + st.at) * p.V;
  const int off = (int)(rp & (N - 1));
  const int64_t v0 = (int64_t)c * kSvThreads * kSvVecs;
  SvVec<DT> x[VECS], y[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int64_t e0 = (v0 + i * kSvRest + tid) * N - off;
    x[i] = sv_load<DT>(p.logits, rp, e0, p.V);
    y[i] = sv_load<DT>(p.draft, rq, e0, p.V);
  }
  const SvRow row = sv_combine(p.rec + sv_rec_at(p, b, st.at, st.depth, p.T), p.S, h);
  const SvRow rowq = sv_combine(p.rec_q + sv_rec_at(p, b, st.at, st.depth, p.T - 1), p.S, h);
  const double zp = 1.0 / row.Z, zq = 1.0 / rowq.Z;
  const double mp = row.M * h.s, mq = rowq.M * h.s;
  double z = 0.0;
  if (fabs(mp) < 1024.0 && fabs(mq) < 1024.0 && row.M < kSvTop && rowq.M < kSvTop) {
    // as in sv_sum; a pair of least weights (2^-1000) adds nothing
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e)
        z += fmax(sv_exp2_fast(fma((double)x[i].raw(e), h.s, -mp)) * zp -
                      sv_exp2_fast(fma((double)y[i].raw(e), h.s, -mq)) * zq,
                  0.0);
  } else {
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e)
        z += fmax(sv_exp2(((double)x[i].at(e) - row.M) * h.s) * zp -
                      sv_exp2(((double)y[i].at(e) - rowq.M) * h.s) * zq,
                  0.0);
  }
  z = wave_sum(z);
  if ((tid & 63) == 0) s_s[wave] = z;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < NW; ++i) z += s_s[i];
    p.rest[b * p.S + c] = z;
  }
}

// Chains: the next token.
template <int DT>
__global__ __launch_bounds__(kSvFinish) void sv_chain_finish_kernel(SvParams p) {
  constexpr int NT = kSvFinish;
  __shared__ SvDraw<NT> dr;
  const int64_t b = blockIdx.x;
  const SvState st = p.state[(int64_t)(p.L + 1) * p.batch + b];
  const SvHeat h = sv_heat(p, b);
  const int d = st.depth;
  const SvRec* rec = p.rec + sv_rec_at(p, b, st.at, d, p.T);
  const SvRow row = sv_combine(rec, p.S, h);
  const int64_t rp = (b * p.T + st.at) * p.V;
  int token = -1;
  double w = 0.0;
  if (row.Z > 0.0 && row.greedy) {
    token = row.arg;
    w = 1.0;
  } else if (row.Z > 0.0) {
    const double u = sv_uniform(p, b, p.L);
    if (st.done == 2) {
      const SvRow rowq = sv_combine(p.rec_q + sv_rec_at(p, b, st.at, d, p.T - 1), p.S, h);
      for (int c = threadIdx.x; c < p.S; c += NT) dr.rest[c] = p.rest[b * p.S + c];
      __syncthreads();
      double total = 0.0;
      for (int c = 0; c < p.S; ++c) total += dr.rest[c];
      if (total > 0.0 && rowq.Z > 0.0)
        token = sv_draw<DT, true, NT>(p, rp, (b * (p.T - 1) + st.at) * p.V, row, rowq, nullptr, 0,
                                      u * total, dr);
    }
    if (token < 0) {  // the whole chain stands, or p = q
      __syncthreads();
      for (int c = threadIdx.x; c < p.S; c += NT)
        dr.rest[c] = rec[c].sum * sv_exp2(((double)rec[c].mx - row.M) * row.s);
      __syncthreads();
      token = sv_draw<DT, false, NT>(p, rp, 0, row, row, nullptr, 0, u * row.Z, dr);
    }
    if (token >= 0) w = row.weight(sv_logit<DT>(p.logits, rp, token), token);
  }
  sv_tail<true>(p, b, d, token, w, row.Z);
}

}  // namespace ddt
