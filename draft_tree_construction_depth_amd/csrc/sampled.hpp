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
// FMA at the rate of an unpacked float32 one; exp2 is a degree-11 polynomial.
//
// The row sums (records) are formed by workgroups of 256 threads, each over a
// chunk of 8 16-byte vectors per thread held in registers: its maximum, then
// the sum of its weights against that maximum. Only the rows on the path
// matter, but which they are is known only step by step; the host picks one
// of two schedules (accept_plan in api.hip).
#pragma once

#include "common.hpp"

namespace ddt {

constexpr int kSvThreads = 256;
constexpr int kSvVecs = 8;       // 16-byte vectors per thread and chunk
constexpr int kSvMaxS = 512;     // chunks per row
constexpr int kSvMaxB = 512;     // nodes
constexpr int kSvChunkMax = kSvThreads * kSvVecs * 8;  // elements (bf16)

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
  int32_t S;    // chunks per row
  int32_t stepped;
  SvRec* rec;      // all rows: [batch][T][S]; stepped: [2][batch][S]
  SvRec* rec_q;    // chains: the same of the drafter's rows
  SvState* state;  // stepped: [L+2][batch]; else [1][batch]
  double* rest;    // chains: [batch][S] sums of max(0, p - q)
};

typedef unsigned int sv_u32x4 __attribute__((ext_vector_type(4)));

template <int DT>
struct SvVec {
  static constexpr int N = DT == 0 ? 8 : 4;  // elements of a 16-byte vector
  sv_u32x4 r;
  // element e; NaN counts as -inf, +inf as the largest finite value
  __device__ __forceinline__ float at(int e) const {
    const float x = DT == 0 ? __uint_as_float(e & 1 ? r[e >> 1] & 0xFFFF0000u : r[e >> 1] << 16)
                            : __uint_as_float(r[e & 3]);
    return x == x ? fminf(x, 3.402823466e38f) : -INFINITY;
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
// Taylor polynomial of exp on [-ln2/2, ln2/2], whose first term left out is
// below 7e-15 of the result.
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

// Inclusive scan of one double per lane over the wave (every lane active).
__device__ __forceinline__ double wave_incl_scan_f64(double x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
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

// Combines a row's S records; every wave does it for itself.
__device__ __forceinline__ SvRow sv_combine(const SvRec* rec, int S, const SvHeat& h) {
  const int lane = threadIdx.x & 63;
  float m = -INFINITY;
  for (int c = lane; c < S; c += kWave) m = fmaxf(m, rec[c].mx);
  m = wave_max(m);
  double z = 0.0;
  int arg = 0x7FFFFFFF;
  for (int c = lane; c < S; c += kWave) {
    const SvRec r = rec[c];
    z += r.sum * sv_exp2(((double)r.mx - (double)m) * h.s);
    if (r.mx == m && r.arg < arg) arg = r.arg;
  }
  SvRow row;
  row.M = (double)m;
  row.s = h.s;
  row.greedy = h.greedy;
  const bool any = m > -INFINITY;
  z = wave_sum(z);
  row.Z = !any ? 0.0 : (h.greedy ? 1.0 : z);
  row.arg = any && h.greedy ? wave_min(arg) : -1;
  return row;
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
    for (int e = 0; e < N; ++e) m = fmaxf(m, x[i].at(e));
  m = wave_max(m);
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
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kSvVecs; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) z += sv_exp2(((double)x[i].at(e) - (double)m) * h.s);
    z = wave_sum(z);
    if ((tid & 63) == 0) s_s[w] = z;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < NW; ++i) z += s_s[i];
      *out = SvRec{m > -INFINITY ? z : 0.0, m, 0x7FFFFFFF};
    }
  }
}

// Records of every row (of the drafter's rows too, for chains).
template <int DT, bool CHAIN>
__global__ __launch_bounds__(kSvThreads) void sv_rows_kernel(SvParams p) {
  const int64_t id = blockIdx.x;
  const int c = (int)(id % p.S);
  int64_t row = id / p.S;
  const bool q = CHAIN && row >= p.batch * p.T;
  if (q) row -= p.batch * p.T;
  const int per = q ? p.T - 1 : p.T;
  const int64_t b = row / per;
  const int i = (int)(row - b * per), n = sv_count(p, b);
  if (i > n || (q && i >= n)) return;
  sv_chunk<DT>(q ? p.draft : p.logits, row * p.V, p.V, c, sv_heat(p, b),
               (q ? p.rec_q : p.rec) + row * p.S + c);
}

// LDS of a decision and of the final draw.
struct SvShared {
  double w[kSvMaxB];
  int tok[kSvMaxB];
  int pick;
  int n;
  double edge;
  double z;
  double seg[kSvVecs][kSvThreads / kWave];
  uint32_t bits[kSvChunkMax / 32];
  int found;
  int last;
  double rest[kSvMaxS];
};

// The tree's decision at one node: the child that t = u Z falls on (-1: none),
// and the children's total weight. The tokens of the children that take a
// part of the line are left in sh.tok[0 .. sh.n). Every thread calls it.
template <int DT>
__device__ int sv_decide_tree(const SvParams& p, int64_t b, int node, int d, const SvRow& row,
                              SvShared& sh, double& t, double& edge, double& wt) {
  const int n = d < p.L ? sv_count(p, b) : 0;
  const int B = p.T - 1, tid = threadIdx.x, lane = tid & 63;
  const int64_t r0 = (b * p.T + node) * p.V;
  t = sv_uniform(p, b, d) * row.Z;
  __syncthreads();
  for (int j = tid; j < n; j += kSvThreads) {
    int tok = -1;
    if (p.parents[b * B + j] == node && node <= j) {
      tok = p.tokens[b * B + j];
      if (tok < 0 || tok >= p.V) tok = -1;
    }
    sh.tok[j] = tok;
    sh.w[j] = tok >= 0 ? row.weight(sv_logit<DT>(p.logits, r0, tok), tok) : 0.0;
  }
  __syncthreads();
  // a token that an earlier sibling carries already takes no second part
  bool dup[2] = {false, false};
  for (int q = 0; q < 2; ++q) {
    const int j = tid + q * kSvThreads;
    if (j < n && sh.tok[j] >= 0)
      for (int i = 0; i < j; ++i) dup[q] |= sh.tok[i] == sh.tok[j];
  }
  __syncthreads();
  for (int q = 0; q < 2; ++q) {
    const int j = tid + q * kSvThreads;
    if (dup[q]) {
      sh.tok[j] = -1;
      sh.w[j] = 0.0;
    }
  }
  __syncthreads();
  if (tid < kWave) {
    double base = 0.0;
    int pick = -1, kept = 0;
    for (int j0 = 0; j0 < n; j0 += kWave) {
      const int j = j0 + lane;
      const int tok = j < n ? sh.tok[j] : -1;
      const uint64_t kids = __ballot(tok >= 0);
      if (!kids) continue;
      const double cum = base + wave_incl_scan_f64(j < n ? sh.w[j] : 0.0);
      const uint64_t hit = __ballot(tok >= 0 && t < cum);
      if (hit && pick < 0) pick = j0 + __builtin_ctzll(hit);
      base = __shfl(cum, 63);
      if (tok >= 0) sh.tok[kept + lanes_below(kids)] = tok;  // never ahead of the reads
      kept += __popcll(kids);
    }
    if (lane == 0) {
      sh.pick = pick;
      sh.edge = base;
      sh.n = kept;
      sh.z = pick >= 0 ? sh.w[pick] : 0.0;
    }
  }
  __syncthreads();
  edge = sh.edge;
  wt = sh.z;
  return sh.pick;
}

__device__ __forceinline__ float sv_logp(double w, double Z) {
  return Z > 0.0 ? (float)(log(w) - log(Z)) : -INFINITY;
}

// Draws from the weights of a chunk (minus q's for PQ, without the tokens
// marked in sh.bits): the first element whose running sum passes t, else the
// last with any weight, else -1. w_out: its weight. Every thread calls it.
template <int DT, bool PQ>
__device__ int sv_draw_chunk(const SvParams& p, int64_t rp, int64_t rq, int c, const SvRow& row,
                             const SvRow& rowq, bool marked, double t, SvShared& sh, double& w_out) {
  constexpr int N = SvVec<DT>::N, NW = kSvThreads / kWave;
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int64_t v0 = (int64_t)c * kSvThreads * kSvVecs;
  const int off = (int)(rp & (N - 1));
  const double zp = 1.0 / row.Z, zq = PQ ? 1.0 / rowq.Z : 0.0;
  SvVec<DT> x[kSvVecs], y[PQ ? kSvVecs : 1];
  double incl[kSvVecs];
  auto weight = [&](int i, int e) -> double {
    const int64_t id = (v0 + i * kSvThreads + tid) * N - off + e;
    if (id < 0 || id >= p.V) return 0.0;
    double a = row.weight(x[i].at(e), id);
    if (PQ) a = fmax(a * zp - rowq.weight(y[PQ ? i : 0].at(e), id) * zq, 0.0);
    const int k = (int)(id + off - v0 * N);
    if (marked && (sh.bits[k >> 5] >> (k & 31)) & 1) a = 0.0;
    return a;
  };
#pragma unroll
  for (int i = 0; i < kSvVecs; ++i) {
    const int64_t e0 = (v0 + i * kSvThreads + tid) * N - off;
    x[i] = sv_load<DT>(p.logits, rp, e0, p.V);
    if (PQ) y[PQ ? i : 0] = sv_load<DT>(p.draft, rq, e0, p.V);
  }
  if (tid == 0) sh.found = sh.last = -1;
  int last = -1;
#pragma unroll
  for (int i = 0; i < kSvVecs; ++i) {
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const double a = weight(i, e);
      sum += a;
      if (a > 0.0) last = i * N + e;
    }
    incl[i] = wave_incl_scan_f64(sum);
    if (lane == 63) sh.seg[i][w] = incl[i];
  }
  __syncthreads();
  double run = 0.0;
  int hit = -1;
  for (int g = 0; g < kSvVecs * NW; ++g) {
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
      for (int i = 0; i < kSvVecs; ++i) {
        if (i != hit / NW) continue;
        const uint64_t over = __ballot(run + incl[i] > t);
        const int l = __builtin_ctzll(over);
        const double before = __shfl_up(incl[i], 1);
        if (lane == l) {
          double cum = run + (lane > 0 ? before : 0.0);
          int at = -1;
          double wa = 0.0;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const double a = weight(i, e);
            const bool open = at < 0 || !(cum > t);
            cum += a;
            if (a > 0.0 && open) {
              at = e;
              wa = a;
            }
          }
          sh.found = (int)((v0 + i * kSvThreads + tid) * N - off) + at;
          sh.z = wa;
        }
      }
    }
    __syncthreads();
  } else {
    // the last element with any weight
    const int id = last < 0 ? -1
                            : (int)((v0 + (last / N) * kSvThreads + tid) * N - off) + last % N;
    const int top = wave_max(id);
    if (lane == 0) atomicMax(&sh.last, top);
    __syncthreads();
    const int pickid = sh.last;
    if (pickid >= 0 && pickid == id) {
#pragma unroll
      for (int i = 0; i < kSvVecs; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (i * N + e == last) sh.z = weight(i, e);
    }
    if (tid == 0) sh.found = pickid;
    __syncthreads();
  }
  const int found = sh.found;
  w_out = sh.z;
  __syncthreads();
  return found;
}

// Draws the next token from a row whose chunk sums are sh.rest[0 .. S): the
// chunk that t falls into, then the element; where rounding leaves no weight
// there, the chunks behind it, then those before it. Every thread calls it.
template <int DT, bool PQ>
__device__ int sv_draw(const SvParams& p, int64_t rp, int64_t rq, const SvRow& row,
                       const SvRow& rowq, int n_marked, double t, SvShared& sh, double& w_out) {
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
      for (int i = tid; i < kSvChunkMax / 32; i += kSvThreads) sh.bits[i] = 0;
      __syncthreads();
      for (int i = tid; i < n_marked; i += kSvThreads) {
        const int64_t k = (int64_t)sh.tok[i] + off - (int64_t)c * kSvThreads * kSvVecs * N;
        if (k >= 0 && k < kSvThreads * kSvVecs * N)
          atomicOr(&sh.bits[k >> 5], 1u << (k & 31));
      }
      __syncthreads();
    }
    const int id = sv_draw_chunk<DT, PQ>(p, rp, rq, c, row, rowq, n_marked > 0, tc, sh, w_out);
    if (id >= 0) return id;
  }
  return -1;
}

// Where the records of a row lie: by row, or (stepped) by request and the
// parity of the depth.
__device__ __forceinline__ int64_t sv_rec_at(const SvParams& p, int64_t b, int at, int d, int per) {
  return p.stepped ? ((int64_t)(d & 1) * p.batch + b) * p.S : (b * per + at) * p.S;
}

// A chain's test of guess d at row d: true where it stands.
template <int DT>
__device__ bool sv_decide_chain(const SvParams& p, int64_t b, int d, const SvRow& row,
                                const SvRow& rowq, double& wt) {
  const int P = p.T - 1;
  const int x = p.tokens[b * P + d];
  wt = 0.0;
  if (x < 0 || x >= p.V) return false;
  const double wp = row.weight(sv_logit<DT>(p.logits, (b * p.T + d) * p.V, x), x);
  const double wq = rowq.weight(sv_logit<DT>(p.draft, (b * P + d) * p.V, x), x);
  wt = wp;
  // (a drafter's row with every token masked has q = 0)
  return sv_uniform(p, b, d) * wq * row.Z < wp * (rowq.Z > 0.0 ? rowq.Z : 1.0);
}

// One decision at (st.at, st.depth), whose row's records are complete:
// advances st, or marks it done. Writes the accepted node and its
// log-probability where `write`.
template <int DT, bool CHAIN>
__device__ void sv_advance(const SvParams& p, int64_t b, SvState& st, bool write, SvShared& sh,
                           SvRow& row, SvRow& rowq, double& t, double& edge) {
  const SvHeat h = sv_heat(p, b);
  const int d = st.depth, P = p.T - 1;
  row = sv_combine(p.rec + sv_rec_at(p, b, st.at, d, p.T), p.S, h);
  double wt = 0.0;
  int next = -1;
  if (CHAIN) {
    if (d < sv_count(p, b)) {
      rowq = sv_combine(p.rec_q + sv_rec_at(p, b, d, d, P), p.S, h);
      if (sv_decide_chain<DT>(p, b, d, row, rowq, wt)) next = d + 1;
      else st.done = 2;
    } else {
      st.done = 1;
    }
  } else {
    const int pick = sv_decide_tree<DT>(p, b, st.at, d, row, sh, t, edge, wt);
    if (pick >= 0) next = pick + 1;
    else st.done = 1;
  }
  if (next >= 0) {
    if (write && threadIdx.x == 0) {
      if (!CHAIN) p.accepted[b * p.L + d] = next;
      if (p.logp) p.logp[b * (p.L + 1) + d] = sv_logp(wt, row.Z);
    }
    st.at = next;
    st.depth = d + 1;
  }
}

// One step of the walk for every request: the decision at the row whose
// records the step before formed, then one chunk of the next row's records.
template <int DT, bool CHAIN>
__global__ __launch_bounds__(kSvThreads) void sv_step_kernel(SvParams p, int step) {
  __shared__ SvShared sh;
  const int64_t id = blockIdx.x;
  const int64_t per = CHAIN ? 2 * (int64_t)p.S : p.S;
  const int64_t b = id / per;
  int c = (int)(id - b * per);
  const bool q = CHAIN && c >= p.S;
  const bool first = c == 0;
  if (q) c -= p.S;
  SvState st{0, 0, 0, 0};
  if (step > 0) {
    st = p.state[(int64_t)(step - 1) * p.batch + b];
    if (!st.done) {
      SvRow row, rowq;
      double t, edge;
      sv_advance<DT, CHAIN>(p, b, st, first, sh, row, rowq, t, edge);
    }
  }
  if (first && threadIdx.x == 0) p.state[(int64_t)step * p.batch + b] = st;
  if (st.done || (q && st.at >= sv_count(p, b))) return;
  const int64_t row = b * (q ? p.T - 1 : p.T) + st.at;
  sv_chunk<DT>(q ? p.draft : p.logits, row * p.V, p.V, c, sv_heat(p, b),
               (q ? p.rec_q : p.rec) + ((int64_t)(step & 1) * p.batch + b) * p.S + c);
}

template <int DT, bool CHAIN>
__device__ void sv_tail(const SvParams& p, int64_t b, const SvState& st, int token, double w,
                        double Z) {
  for (int i = st.depth + threadIdx.x; i <= p.L; i += kSvThreads) {
    if (!CHAIN && i < p.L) p.accepted[b * p.L + i] = -1;
    if (p.logp) p.logp[b * (p.L + 1) + i] = i > st.depth ? 0.0f : (token < 0 ? -INFINITY : sv_logp(w, Z));
  }
  if (threadIdx.x == 0) {
    p.accept_len[b] = st.depth;
    p.next_token[b] = token;
  }
}

// Trees: the rest of the walk and the next token, one workgroup per request.
template <int DT>
__global__ __launch_bounds__(kSvThreads) void sv_finish_kernel(SvParams p, int step) {
  __shared__ SvShared sh;
  const int64_t b = blockIdx.x;
  SvState st{0, 0, 0, 0};
  if (p.stepped) st = p.state[(int64_t)step * p.batch + b];
  SvRow row, rowq;
  double t = 0.0, edge = 0.0;
  st.done = 0;  // a decision that ended the walk is made again, for its line
  while (!st.done) sv_advance<DT, false>(p, b, st, true, sh, row, rowq, t, edge);
  const int n = sh.n;
  int token = -1;
  double w = 0.0;
  if (row.greedy) {
    token = row.arg;
    w = 1.0;
  } else if (row.Z > 0.0) {
    // the chunks' weights without the children's
    const SvRec* rec = p.rec + sv_rec_at(p, b, st.at, st.depth, p.T);
    const int64_t r0 = (b * p.T + st.at) * p.V;
    constexpr int N = SvVec<DT>::N;
    const int off = (int)(r0 & (N - 1));
    for (int i = threadIdx.x; i < n; i += kSvThreads)
      sh.w[i] = row.weight(sv_logit<DT>(p.logits, r0, sh.tok[i]), sh.tok[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < p.S; c += kSvThreads) {
      double s = rec[c].sum * sv_exp2(((double)rec[c].mx - row.M) * row.s);
      for (int i = 0; i < n; ++i)
        if ((sh.tok[i] + off) / (kSvThreads * kSvVecs * N) == c) s -= sh.w[i];
      sh.rest[c] = fmax(s, 0.0);
    }
    __syncthreads();
    token = sv_draw<DT, false>(p, r0, 0, row, row, n, t - edge, sh, w);
  }
  sv_tail<DT, false>(p, b, st, token, w, row.Z);
}

// Chains: the rest of the walk.
template <int DT>
__global__ __launch_bounds__(kSvThreads) void sv_chain_walk_kernel(SvParams p, int step) {
  __shared__ SvShared sh;
  const int64_t b = blockIdx.x;
  SvState st{0, 0, 0, 0};
  if (p.stepped) st = p.state[(int64_t)step * p.batch + b];
  SvRow row, rowq;
  double t, edge;
  while (!st.done) sv_advance<DT, true>(p, b, st, true, sh, row, rowq, t, edge);
  if (threadIdx.x == 0) p.state[(int64_t)(p.stepped ? step + 1 : 0) * p.batch + b] = st;
}

// Chains: chunk sums of max(0, p - q) where a guess fell.
template <int DT>
__global__ __launch_bounds__(kSvThreads) void sv_chain_rest_kernel(SvParams p, int step) {
  constexpr int N = SvVec<DT>::N, NW = kSvThreads / kWave;
  __shared__ double s_s[NW];
  const int64_t b = blockIdx.x / p.S;
  const int c = (int)(blockIdx.x - b * p.S), tid = threadIdx.x;
  const SvState st = p.state[(int64_t)step * p.batch + b];
  const SvHeat h = sv_heat(p, b);
  if (st.done != 2 || h.greedy) return;
  const int64_t rp = (b * p.T + st.at) * p.V, rq = (b * (p.T - 1) + st.at) * p.V;
  const int off = (int)(rp & (N - 1));
  const int64_t v0 = (int64_t)c * kSvThreads * kSvVecs;
  SvVec<DT> x[kSvVecs], y[kSvVecs];
#pragma unroll
  for (int i = 0; i < kSvVecs; ++i) {
    const int64_t e0 = (v0 + i * kSvThreads + tid) * N - off;
    x[i] = sv_load<DT>(p.logits, rp, e0, p.V);
    y[i] = sv_load<DT>(p.draft, rq, e0, p.V);
  }
  const SvRow row = sv_combine(p.rec + sv_rec_at(p, b, st.at, st.depth, p.T), p.S, h);
  const SvRow rowq = sv_combine(p.rec_q + sv_rec_at(p, b, st.at, st.depth, p.T - 1), p.S, h);
  const double zp = 1.0 / row.Z, zq = 1.0 / rowq.Z;
  double z = 0.0;
#pragma unroll
  for (int i = 0; i < kSvVecs; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e)
      z += fmax(sv_exp2(((double)x[i].at(e) - row.M) * h.s) * zp -
                    sv_exp2(((double)y[i].at(e) - rowq.M) * h.s) * zq,
                0.0);
  z = wave_sum(z);
  if ((tid & 63) == 0) s_s[tid >> 6] = z;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < NW; ++i) z += s_s[i];
    p.rest[b * p.S + c] = z;
  }
}

// Chains: the next token.
template <int DT>
__global__ __launch_bounds__(kSvThreads) void sv_chain_finish_kernel(SvParams p, int step) {
  __shared__ SvShared sh;
  const int64_t b = blockIdx.x;
  const SvState st = p.state[(int64_t)step * p.batch + b];
  const SvHeat h = sv_heat(p, b);
  const int d = st.depth;
  const SvRec* rec = p.rec + sv_rec_at(p, b, st.at, d, p.T);
  const SvRow row = sv_combine(rec, p.S, h);
  const int64_t rp = (b * p.T + st.at) * p.V;
  int token = -1;
  double w = 0.0;
  if (row.greedy) {
    token = row.arg;
    w = 1.0;
  } else if (row.Z > 0.0) {
    const double u = sv_uniform(p, b, p.L);
    if (st.done == 2) {
      const SvRow rowq = sv_combine(p.rec_q + sv_rec_at(p, b, st.at, d, p.T - 1), p.S, h);
      for (int c = threadIdx.x; c < p.S; c += kSvThreads) sh.rest[c] = p.rest[b * p.S + c];
      __syncthreads();
      double total = 0.0;
      for (int c = 0; c < p.S; ++c) total += sh.rest[c];
      if (total > 0.0 && rowq.Z > 0.0)
        token = sv_draw<DT, true>(p, rp, (b * (p.T - 1) + st.at) * p.V, row, rowq, 0, u * total,
                                  sh, w);
    }
    if (token < 0) {  // the whole chain stands, or p = q
      __syncthreads();
      for (int c = threadIdx.x; c < p.S; c += kSvThreads)
        sh.rest[c] = rec[c].sum * sv_exp2(((double)rec[c].mx - row.M) * row.s);
      __syncthreads();
      token = sv_draw<DT, false>(p, rp, 0, row, row, 0, u * row.Z, sh, w);
    }
    if (token >= 0) w = row.weight(sv_logit<DT>(p.logits, rp, token), token);
  }
  sv_tail<DT, true>(p, b, st, token, w, row.Z);
}

}  // namespace ddt
