// Log probabilities of given tokens with entropy and top alternatives, and
// their gradient (include/rxl.h: rxl_token_logprob_*).
//
// Forward. Memory-bound: a row of logits is read once. Every thread keeps a
// running maximum m with S = sum 2^y and T = sum 2^y y over what it has seen,
// y = x log2(e) - Y, Y = m log2(e) rounded: one fused operation with one
// rounding. Y's own rounding is in S and T; beyond 2^24, where it would be more
// than 1, y = (x - m) log2(e). When a group of vectors raises Y by d, S and T
// become f S and f (T - d S) with f = 2^-d. From the joined values
// lse = ln2 (Y + log2 S) and entropy = ln2 (log2 S - T / S). On packed pairs
// that is about five issue slots an element, of the eleven that one has at
// the card's copy rate in bf16.
//
// The alternatives cost no second pass: the threads' maxima give a bound that
// enough elements reach. Threads also keep the maximum of every few vectors
// (a slot), and only slots above the bound are read again, from the caches:
// a dozen for eight alternatives.
//
// A row goes to 8 or 16 lanes or to a warp (short rows, no barriers), to a
// block of 64 to 512 threads, or to a cluster of blocks whose results meet in
// the first one's shared memory (a few very long rows).
//
// Measured (the card copies at 6.78 TB/s), bf16: 8192 x 50021 125 us without
// alternatives (6.6 TB/s) and 147 us with 8 (5.6): the bound costs 6, the list
// of slots 6, reading them 7, placing the candidates 2, issue slots are 68%
// busy; 32768 x 8192 83 and 110 us. 65536 x 256 f32 16 and (with 5) 31 us: a
// row's fixed work is as long as its sum. 4 x 32000 with 20 alternatives 6.3 us.
//
// Backward. One pass, a vector in and a vector out: 8192 x 50021 bf16 248 us
// (6.6 TB/s), 1000 x 10007 f32 13.8 us (5.8).
#include <float.h>
#include <math.h>

#include "sm103.cuh"
#include "stream_common.cuh"
#include "train.cuh"

namespace rxl {
namespace {

using namespace stream;
using sm103::griddep_launch_dependents;
using sm103::griddep_wait;

typedef unsigned long long Key;

// Order of values as unsigned integers, all above 0; -0 and +0 are equal.
__device__ __forceinline__ unsigned ordered(float v) {
  const unsigned u = __float_as_uint(v + 0.f);
  return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned o) {
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
// The next float above (of -inf: the lowest finite one).
__device__ __forceinline__ float next_up(float v) { return value_of(ordered(v) + 1); }
// Order of the alternatives: value, then the lower index. Keys of one row are
// distinct, and none is 0.
__device__ __forceinline__ Key key_of(float v, int j) { return ((Key)ordered(v) << 32) | (unsigned)~j; }
__device__ __forceinline__ float value_of(Key k) { return value_of((unsigned)(k >> 32)); }
__device__ __forceinline__ int index_of(Key k) { return (int)~(unsigned)k; }

// ------------------------------------------------------ the running softmax

struct Running {
  float m;    // maximum of what was seen (NaN aside)
  Pair s, t;  // sums of 2^y and 2^y y, in two halves
  __device__ __forceinline__ Running() : m(-INFINITY), s(0.f, 0.f), t(0.f, 0.f) {}
};

// What a maximum's sums are relative to, in powers of two. Near zero it is Y,
// the rounded product, the same wherever it is formed (a product contracted
// into what follows would move Y by up to half its last place, and the sums by
// 2 to that power): at most 1 from m log2(e). Far from zero that distance would
// grow with m until 2^y overflows or vanishes at the maximum itself (half a
// place of Y at 1e10 is 512), so there it is m log2(e) itself, which no float
// has to hold: y comes from the difference x - m. Masks of -1e9 and the like are
// far, and so is a maximum that is infinite.
__device__ __forceinline__ float scaled(float m) { return __fmul_rn(m, kLog2e); }
__device__ __forceinline__ bool near_zero(float m) { return fabsf(m) < 0x1p24f; }

// Brings the sums from r.m to m, which is larger. d: how far the references
// lie apart, the difference of two Y, or of two maxima, or of a Y and a
// maximum. Infinite where a maximum is; then 2^-d is 0. (By cases, of which the
// first two near zero are the usual one: clusters 2 to 4% slower.)
__device__ __forceinline__ void rescale(Running &r, float m) {
  const bool near = near_zero(m), was = near_zero(r.m);
  const float d = fmaf((near ? 0.f : m) - (was ? 0.f : r.m), kLog2e, (near ? scaled(m) : 0.f) - (was ? scaled(r.m) : 0.f));
  const float f = ex2(-d);
  float s0, s1, t0, t1;
  r.s.get(s0, s1);
  r.t.get(t0, t1);
  r.t = Pair(f > 0.f ? f * (t0 - d * s0) : 0.f, f > 0.f ? f * (t1 - d * s1) : 0.f);
  r.s = Pair(s0 * f, s1 * f);  // NaN stays
  r.m = m;
}

// Adds two values of which neither is above the maximum: y = x log2(e) + neg,
// clamped where 2^y is 0 (-inf included), so that 2^y y is 0 there, too.
__device__ __forceinline__ void take2(Running &r, Pair x, Pair c, Pair neg, bool clamp) {
  Pair y = fma(x, c, neg);
  float a, b;
  y.get(a, b);
  if (clamp) {
    a = max_nan(a, -150.f);
    b = max_nan(b, -150.f);
    y = Pair(a, b);
  }
  const Pair e(ex2(a), ex2(b));
  r.s = add(r.s, e);
  r.t = fma(e, y, r.t);
}

__device__ __forceinline__ float max_of(const uint4 &w, __nv_bfloat16) {
  const __nv_bfloat162 a = *(const __nv_bfloat162 *)&w.x, b = *(const __nv_bfloat162 *)&w.y,
                       c = *(const __nv_bfloat162 *)&w.z, d = *(const __nv_bfloat162 *)&w.w;
  const __nv_bfloat162 m = __hmax2(__hmax2(a, b), __hmax2(c, d));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float max_of(const uint4 &w, float) {
  return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
// A vector of -inf.
__device__ __forceinline__ uint4 nothing(__nv_bfloat16) { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
__device__ __forceinline__ uint4 nothing(float) { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }

// x - m for a maximum far from zero. Nothing but -inf (m = -inf) is as far
// below the lowest float. Two bf16 values that far from zero are equal or at
// least 2^16 apart, so that rounding the difference to bf16 changes no 2^y.
__device__ __forceinline__ float from_far(float x, float m) { return x - fmaxf(m, -FLT_MAX); }
__device__ __forceinline__ uint4 from_far(const uint4 &w, float m, float) {
  return make_uint4(__float_as_uint(from_far(__uint_as_float(w.x), m)), __float_as_uint(from_far(__uint_as_float(w.y), m)),
                    __float_as_uint(from_far(__uint_as_float(w.z), m)), __float_as_uint(from_far(__uint_as_float(w.w), m)));
}
__device__ __forceinline__ uint4 from_far(const uint4 &w, float m, __nv_bfloat16) {
  const __nv_bfloat162 base = __float2bfloat162_rn(fmaxf(m, -0x1.FEp127f));
  uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 d = __hsub2(*(const __nv_bfloat162 *)&u[i], base);
    u[i] = *(const uint32_t *)&d;
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// bf16 logits are clamped as they come, two at a time: -2^100 is far enough
// below a maximum near zero, and below the difference from one far from it.
__device__ __forceinline__ void take_vector(Running &r, const uint4 &w, Pair c, Pair neg, __nv_bfloat16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  const __nv_bfloat162 low = __floats2bfloat162_rn(-0x1p100f, -0x1p100f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __hmax2_nan(*(const __nv_bfloat162 *)&u[i], low);
    const uint32_t x = *(const uint32_t *)&b;
    take2(r, Pair(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)), c, neg, false);
  }
}
__device__ __forceinline__ void take_vector(Running &r, const uint4 &w, Pair c, Pair neg, float) {
  take2(r, Pair(__uint_as_float(w.x), __uint_as_float(w.y)), c, neg, true);
  take2(r, Pair(__uint_as_float(w.z), __uint_as_float(w.w)), c, neg, true);
}

// Adds N vectors, of which `top` receives the maxima; the largest of them.
template <typename T, int N>
__device__ __forceinline__ float take(Running &r, const uint4 (&w)[N], float (&top)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) top[k] = max_of(w[k], T());
  float g = top[0];
#pragma unroll
  for (int k = 1; k < N; ++k) g = fmaxf(g, top[k]);
  if (g > r.m) rescale(r, g);
  // (one loop over values that are from_far already, or not: 65536 x 1000 bf16 32
  // us, 28.6 so)
  const Pair c(kLog2e, kLog2e);
  if (near_zero(r.m)) {
    const float y = -scaled(r.m);
    const Pair neg(y, y);
#pragma unroll
    for (int k = 0; k < N; ++k) take_vector(r, w[k], c, neg, T());
  } else {
    const Pair neg(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < N; ++k) take_vector(r, from_far(w[k], r.m, T()), c, neg, T());
  }
  return g;
}
// Adds one value.
__device__ __forceinline__ void take(Running &r, float x) {
  if (x > r.m) rescale(r, x);
  const bool near = near_zero(r.m);
  const float y = near ? -scaled(r.m) : 0.f;
  take2(r, Pair(near ? x : from_far(x, r.m), -INFINITY), Pair(kLog2e, kLog2e), Pair(y, y), true);
}

// What a row's results are made of.
struct Outputs {
  const int32_t *tokens;
  float *logp, *lse, *entropy;
  int32_t *top_ids;
  float *top_logp;
};

// A row's joined sum as its maximum and the log of the sum relative to it.
// lse = m + rest rounds to the place of a maximum far from zero; log p = (x -
// m) - rest does not.
struct Norm {
  float m, rest, l2;  // l2: log2 of the sum
  __device__ __forceinline__ Norm(float max, float s) : m(max) {
    if (m == INFINITY) s = NAN;
    l2 = log2f(s);
    // near zero the sum is relative to the rounded m log2(e): what rounding took off
    const float off = near_zero(m) ? fmaf(m, kLog2e, -scaled(m)) : 0.f;
    rest = kLn2 * (l2 - off);
  }
  // nothing but -inf: its lse and log probabilities are -inf
  __device__ __forceinline__ bool none() const { return m == -INFINITY && rest == rest; }
  __device__ __forceinline__ float lse() const { return none() ? -INFINITY : m + rest; }
  __device__ __forceinline__ float log_p(float x) const { return none() ? -INFINITY : (x - m) - rest; }
};

// The given token of a row and its logit; read early, by the thread that
// finishes the row. No token: tok -1.
struct Given {
  int tok;
  float x;
  template <typename T>
  __device__ __forceinline__ Given(const Outputs &o, const T *row_x, long long row, int V, bool mine) : tok(-1), x(0.f) {
    if (mine && o.tokens) {
      tok = o.tokens[row];
      if (tok < 0 || tok >= V) tok = -1;
      else x = to_f32(row_x[tok]);
    }
  }
};

// One thread: lse, entropy and the token's log probability.
__device__ __forceinline__ void finish(const Outputs &o, long long row, const Norm &n, float s, float t, const Given &g) {
  o.lse[row] = n.lse();
  if (o.entropy) o.entropy[row] = n.none() ? 0.f : kLn2 * (n.l2 - t / s);
  if (o.tokens) o.logp[row] = g.tok >= 0 ? n.log_p(g.x) : 0.f;
}

// A row's part [begin, end): single elements up to the first 16-byte border,
// whole vectors, single elements (fewer than 2 kVec in all).
template <typename T>
struct Part {
  const T *x;           // the row
  int begin, end;
  int first, vectors;   // element of the first whole vector; their number
  __device__ __forceinline__ Part(const T *row, int b, int e) : x(row), begin(b), end(e) {
    const int off = (int)(((uintptr_t)(row + b) & 15) / sizeof(T));
    first = b + (off ? kVec<T> - off : 0);
    if (first > e) first = e;
    vectors = (e - first) / kVec<T>;
  }
  __device__ __forceinline__ uint4 load(int i) const { return *((const uint4 *)(x + first) + i); }
  __device__ __forceinline__ int singles() const { return (first - begin) + (end - first - vectors * kVec<T>); }
  __device__ __forceinline__ int single(int s) const {
    return s < first - begin ? begin + s : first + vectors * kVec<T> + (s - (first - begin));
  }
};

constexpr int kDeep = 4;  // vectors of a thread in flight: a group

// Threads that share a row part are numbered 0 .. N-1: vector u of thread t.
template <int N>
__device__ __forceinline__ int vector_of(int u, int t) {
  return u * N + t;
}

// A group of a thread's vectors: FULL where the part has all of them.
template <int N, bool FULL, typename T>
__device__ __forceinline__ void load_group(uint4 (&w)[kDeep], const Part<T> &p, int g, int t, bool live = true) {
  const uint4 *at = (const uint4 *)(p.x + p.first) + vector_of<N>(g * kDeep, t);
#pragma unroll
  for (int k = 0; k < kDeep; ++k)
    w[k] = FULL || (live && vector_of<N>(g * kDeep + k, t) < p.vectors) ? at[k * N] : nothing(T());
}

// Which of a vector's elements reach `low`, as bits.
template <typename T>
__device__ __forceinline__ unsigned reaching(const uint4 &w, float low) {
  float x[kVec<T>];
  unpack(w, x);
  unsigned hits = 0;
#pragma unroll
  for (int k = 0; k < kVec<T>; ++k) hits |= x[k] >= low ? 1u << k : 0u;
  return hits;
}
template <typename T>
__device__ __forceinline__ float element(const uint4 &w, int k) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w);
  const uint32_t u = k < 2 ? w.x : k < 4 ? w.y : k < 6 ? w.z : w.w;
  return __uint_as_float(k & 1 ? u & 0xFFFF0000u : u << 16);
}

// Sum of the counts of the lanes before this one, of L lanes; `total`: of all.
template <int L>
__device__ __forceinline__ int lanes_before(int n, int &total) {
  const int lane = (int)threadIdx.x % L;
  int sum = n;
#pragma unroll
  for (int d = 1; d < L; d *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, sum, d, L);
    if (lane >= d) sum += up;
  }
  total = __shfl_sync(0xffffffffu, sum, L - 1, L);
  return sum - n;
}

// ------------------------------------------------- 8 lanes or a warp for a row

constexpr int kShortThreads = 256;
// Blocks on an SM: without alternatives 64 registers a thread are enough;
// with them three blocks and no spills are faster than four (65536 x 1000
// bf16, 4 alternatives: 45 against 58 us).
constexpr int short_blocks(bool top) { return top ? 3 : 4; }
constexpr int kShortKeys = 320;  // a warp's room for candidates

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int k = L / 2; k > 0; k >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int k = L / 2; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}
template <int L>
__device__ __forceinline__ Key lanes_max(Key v) {
#pragma unroll
  for (int k = L / 2; k > 0; k >>= 1) {
    const Key o = __shfl_xor_sync(0xffffffffu, v, k);
    v = o > v ? o : v;
  }
  return v;
}

// A row's shared memory in the short kernel. A lane keeps kSlots maxima, of
// kBy vectors each, and of the vectors kSlots kBy, 2 kSlots kBy .. further on.
template <int L>
struct ShortShared {
  static constexpr int kRoom = kShortKeys * L / 32;
  static constexpr int kSlots = L == 32 ? 8 : 16, kBy = L == 32 ? kDeep : 1;
  float slots[kSlots][L];
  unsigned char list[L * kSlots];  // slots to be read again: lane + L slot
  Key keys[kRoom];
  Key top[kMaxTopK];
  float pad[L];  // a warp's rows lie in banks of their own
};
static_assert(sizeof(ShortShared<8>) % 128 == 32 && sizeof(ShortShared<16>) % 128 == 64, "see pad");

// The n-th largest (from 0) of the lanes' values, two each.
template <int L>
__device__ __forceinline__ float lanes_nth(float a, float b, int n) {
  const int lane = (int)threadIdx.x % L;
  int ra = 0, rb = 1;  // places: by value, then by lane, then a before b (b <= a)
#pragma unroll
  for (int d = 1; d < L; ++d) {
    const float oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
    const bool earlier = (lane ^ d) < lane;
    ra += (oa > a || (oa == a && earlier)) + (ob > a || (ob == a && earlier));
    rb += (oa > b || (oa == b && earlier)) + (ob > b || (ob == b && earlier));
  }
  const int shift = (int)threadIdx.x & 31 & ~(L - 1);
  const unsigned mask = 0xffffffffu >> (32 - L);
  const unsigned in_a = __ballot_sync(0xffffffffu, ra == n) >> shift & mask;
  const unsigned in_b = __ballot_sync(0xffffffffu, rb == n) >> shift & mask;
  const float va = __shfl_sync(0xffffffffu, a, in_a ? __ffs(in_a) - 1 : 0, L);
  const float vb = __shfl_sync(0xffffffffu, b, in_b ? __ffs(in_b) - 1 : 0, L);
  return in_a ? va : vb;
}
// The n-th largest (from 0) of the lanes' values.
template <int L>
__device__ __forceinline__ float lanes_nth(float v, int n) {
  const int lane = (int)threadIdx.x % L;
#pragma unroll
  for (int size = 2; size <= L; size *= 2)
#pragma unroll
    for (int d = size / 2; d > 0; d /= 2) {
      const float o = __shfl_xor_sync(0xffffffffu, v, d);
      const bool larger = ((lane & d) == 0) == ((lane & size) == 0 || size == L);
      v = larger ? fmaxf(v, o) : fminf(v, o);
    }
  return __shfl_sync(0xffffffffu, v, n, L);
}

// The K first alternatives of each of a warp's rows, by the row's L lanes.
// m, m2: the largest and the second largest of the lane's vectors' maxima;
// live: whether the lane has a row. The whole warp calls.
template <typename T, int L>
__device__ __forceinline__ void short_alternatives(ShortShared<L> &sh, const Part<T> &p, float m, float m2, const Norm &norm,
                                                   int K, bool live, const Outputs &o, long long row) {
  constexpr int room = ShortShared<L>::kRoom, S = ShortShared<L>::kSlots, BY = ShortShared<L>::kBy;
  const int lane = (int)threadIdx.x % L;
  // A bound that at least K elements reach: the (K + 1)-th largest of the
  // lanes' maxima, of two each where lanes are few (K < 2 L), which keeps the
  // candidates few. With fewer lanes that have elements, -inf.
  const float bound = L < 32 ? lanes_nth<L>(m, m2, K) : lanes_nth<L>(m, min(L - 1, K));
  // Candidates are what reaches the bound, at least K elements. Where they are
  // too many for the room (ties), or the bound is -inf, only what is above it.
  float low = bound == -INFINITY ? next_up(bound) : bound;
  int count = 0;  // of the row's candidates, the same in its lanes
  bool again = live;
  do {
    if (again) count = 0;
    const auto append = [&](unsigned hits, int j0, const auto &value) {
      int total;
      int at = count + lanes_before<L>(__popc(hits), total);
      for (; hits; hits &= hits - 1, ++at) {
        const int k = __ffs(hits) - 1;
        if (at < room) sh.keys[at] = key_of(value(k), j0 + k);
      }
      count += total;
    };
    unsigned slots = 0;
    if (again && m >= low)
#pragma unroll
      for (int k = 0; k < S; ++k) slots |= sh.slots[k][lane] >= low ? 1u << k : 0u;
    int listed;
    int at = lanes_before<L>(__popc(slots), listed);
    for (; slots; slots &= slots - 1) sh.list[at++] = (unsigned char)(lane + L * (__ffs(slots) - 1));
    __syncwarp();
    const int reads = again ? listed * BY : 0;
    for (int u0 = 0; __any_sync(0xffffffffu, reads > 0 && u0 * L < p.vectors); u0 += S * BY)
      for (int i = lane; __any_sync(0xffffffffu, i - lane < reads); i += L) {
        int v = p.vectors;
        if (i < reads) {
          const int entry = sh.list[i / BY];
          v = vector_of<L>(u0 + entry / L * BY + i % BY, entry % L);
        }
        const uint4 w = v < p.vectors ? p.load(v) : nothing(T());
        append(reaching<T>(w, low), p.first + v * kVec<T>, [&](int k) { return element<T>(w, k); });
      }
    for (int s = lane; __any_sync(0xffffffffu, s - lane < p.singles()); s += L) {
      const bool has = again && s < p.singles();
      const int j = has ? p.single(s) : 0;
      const float v = has ? to_f32(p.x[j]) : -INFINITY;
      append(has && v >= low ? 1u : 0u, j, [&](int) { return v; });
    }
    again = again && count > room && low == bound;
    if (again) low = next_up(bound);
    __syncwarp();
  } while (__any_sync(0xffffffffu, again));
  // Rows made so that a few lanes hold everything large: one sweep for each
  // alternative.
  const bool many = count > room;
  if (__any_sync(0xffffffffu, many)) {
    Key last = ~0ull;
    for (int k = 0; k < K; ++k) {
      Key best = 0;
      if (many)
        for (int e = lane; e < p.end; e += L) {
          const Key c = key_of(to_f32(p.x[e]), e);
          if (c < last && c > best) best = c;
        }
      last = lanes_max<L>(best);
      if (many && lane == 0) sh.top[k] = last;
    }
  }
  // Too few (above the bound, then): the first ones at it, in the row's order.
  const int need = live && !many ? K - count : 0;
  int found = 0;
  for (int base = 0; __any_sync(0xffffffffu, found < need && base < p.end); base += L) {
    const int e = base + lane;
    const bool hit = found < need && e < p.end && to_f32(p.x[e]) == bound;
    int total;
    const int at = found + lanes_before<L>(hit, total);
    if (hit && at < need) sh.keys[count + at] = key_of(bound, e);
    found += total;
  }
  __syncwarp();
  if (live && !many) {
    const int n = count + max(0, min(found, need));
    // distinct keys: a key's place is the number of larger ones
    for (int c = lane; c < n; c += L) {
      const Key key = sh.keys[c];
      int rank = 0;
      for (int i = 0; i < n; ++i) rank += sh.keys[i] > key;
      if (rank < K) sh.top[rank] = key;
    }
    // a row with NaN in it may leave places open
    for (int k = n + lane; k < K; k += L) sh.top[k] = key_of(NAN, k);
  }
  __syncwarp();
  if (live)
    for (int k = lane; k < K; k += L) {
      const Key key = sh.top[k];
      o.top_ids[row * K + k] = index_of(key);
      o.top_logp[row * K + k] = norm.log_p(value_of(key));
    }
  __syncwarp();
}

// Groups of L lanes take rows in turn; the next group of vectors, of this row
// or of the next one, is in flight while one is added. Trip counts are the
// warp's (shuffles need every lane): a lane whose row does not exist adds
// nothing.
template <typename T, int L, bool TOP>
__global__ void __launch_bounds__(kShortThreads, short_blocks(TOP))
logprob_short_kernel(const T *__restrict__ x, long long stride, Outputs o, long long rows, int V, int K) {
  __shared__ ShortShared<L> shared[TOP ? kShortThreads / L : 1];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = (int)threadIdx.x % L, group = (int)threadIdx.x / L;
  ShortShared<L> &sh = shared[TOP ? group : 0];
  constexpr int S = ShortShared<L>::kSlots, BY = ShortShared<L>::kBy;
  static_assert(S * BY % kDeep == 0 && (BY == 1 || BY == kDeep), "a group's maxima go to slots of one turn");
  const long long step = (long long)gridDim.x * (kShortThreads / L);
  long long row = (long long)blockIdx.x * (kShortThreads / L) + group;
  long long first = row - group % (32 / L);  // the warp's first row
  if (first >= rows) return;
  // of every row's vectors; those of one row may be one fewer
  const int groups = (V / kVec<T> + kDeep * L - 1) / (kDeep * L) > 0 ? (V / kVec<T> + kDeep * L - 1) / (kDeep * L) : 1;
  const auto load = [&](uint4 (&w)[kDeep], const Part<T> &p, bool live, int g) {
    if (__all_sync(0xffffffffu, live && (g + 1) * kDeep * L <= p.vectors)) load_group<L, true>(w, p, g, lane);
    else load_group<L, false>(w, p, g, lane, live);
  };
  bool live = row < rows;
  Part<T> p(x + (live ? row : first) * stride, 0, V);
  uint4 next[kDeep];
  load(next, p, live, 0);
#pragma unroll 1
  for (; first < rows; first += step, row += step) {
    const Given given(o, p.x, row, V, live && lane == 0);
    const Part<T> q = p;
    const bool was = live;
    Running r;
    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      uint4 now[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) now[k] = next[k];
      if (g + 1 < groups) {
        load(next, q, was, g + 1);
      } else if (first + step < rows) {
        live = row + step < rows;
        p = Part<T>(x + (live ? row + step : first + step) * stride, 0, V);
        load(next, p, live, 0);
      }
      float top[kDeep];
      const float most = take<T, kDeep>(r, now, top);
      if (TOP) {
#pragma unroll
        for (int k = 0; k < kDeep / BY; ++k) {
          const int u = g * (kDeep / BY) + k;
          const float t = BY == 1 ? top[k] : most;
          if (L < 32) m2 = fmaxf(m2, fminf(m1, t));
          m1 = fmaxf(m1, t);
          sh.slots[u % S][lane] = u < S ? t : fmaxf(t, sh.slots[u % S][lane]);
        }
      }
    }
    if (TOP)
      for (int u = groups * (kDeep / BY); u < S; ++u) sh.slots[u][lane] = -INFINITY;
    for (int s = lane; __any_sync(0xffffffffu, s < q.singles()); s += L)
      if (was && s < q.singles()) take(r, to_f32(q.x[q.single(s)]));
    const float m = lanes_max<L>(r.m);
    if (m > r.m) rescale(r, m);
    float a, b;
    r.s.get(a, b);
    const float sum = lanes_sum<L>(a + b);
    r.t.get(a, b);
    const float t = lanes_sum<L>(a + b);
    const Norm norm(m, sum);
    if (was && lane == 0) finish(o, row, norm, sum, t, given);
    if (TOP) short_alternatives<T, L>(sh, q, m1, m2, norm, K, was, o, row);
  }
}

// ---------------------------------------- a block, or a cluster, for each row

// Maxima a thread keeps, of a group each.
template <int NT>
constexpr int kSlots = NT <= 256 ? 16 : 4096 / NT;
constexpr int kCandidates = 512;     // room for elements above the bound

template <int NT>
struct Shared {
  float warp_m[NT / 32], warp_s[NT / 32], warp_t[NT / 32];
  unsigned best[64];                     // the warps' largest maxima, in order
  int warp_count[NT / 32];
  int count, listed;
  float slots[kSlots<NT>][NT];
  unsigned short list[NT * kSlots<NT>];
  Key keys[kCandidates];
  Key top[kMaxTopK];                     // the part's alternatives in order
  float part[3];                         // the part's maximum and sums
};

// The block's maximum and sums from the threads', the same in every thread,
// and (K > 0) a value that at least K elements of the part reach: the
// (K + 1)-th largest of every warp's j largest among its threads' maxima (the
// last of them, if they are no more than K). Only warps whose lanes all have
// elements take part (the first `full` ones); j makes the values at least
// K + 1. One barrier.
template <int NT>
__device__ __forceinline__ float join(Shared<NT> &sh, Running r, int full, int K, float &m, float &s, float &t) {
  constexpr int kWarps = NT / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float top = r.m;
  m = lanes_max<32>(top);
  if (m > top) rescale(r, m);
  float a, b;
  r.s.get(a, b);
  s = lanes_sum<32>(a + b);
  r.t.get(a, b);
  t = lanes_sum<32>(a + b);
  if (lane == 0) {
    sh.warp_m[warp] = m;
    sh.warp_s[warp] = s;
    sh.warp_t[warp] = t;
  }
  const int j = min(32, K / full + 2), n = j * full;
  if (K && warp < full) {
    unsigned mine = ordered(top);
    for (int k = 0; k < j; ++k) {
      const unsigned v = __reduce_max_sync(0xffffffffu, mine);
      const unsigned who = __ballot_sync(0xffffffffu, mine == v);
      if (lane == __ffs(who) - 1) mine = 0;  // below every value's order
      if (lane == 0) sh.best[warp * j + k] = v;
    }
  }
  if (threadIdx.x == 0) sh.count = sh.listed = 0;
  __syncthreads();
  // each of the first lanes brings one warp's sums to the common maximum
  Running w;
  if (lane < kWarps) {
    w.m = sh.warp_m[lane];
    w.s = Pair(sh.warp_s[lane], 0.f);
    w.t = Pair(sh.warp_t[lane], 0.f);
  }
  m = lanes_max<32>(w.m);
  if (m > w.m) rescale(w, m);
  w.s.get(s, b);
  w.t.get(t, b);
#pragma unroll
  for (int k = kWarps / 2; k > 0; k >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, k);
    t += __shfl_xor_sync(0xffffffffu, t, k);
  }
  s = __shfl_sync(0xffffffffu, s, 0);
  t = __shfl_sync(0xffffffffu, t, 0);
  if (!K) return 0.f;
  // each lane the places of two of the values
  const unsigned v0 = lane < n ? sh.best[lane] : 0, v1 = lane + 32 < n ? sh.best[lane + 32] : 0;
  int r0 = 0, r1 = 0;
  for (int i = 0; i < n; ++i) {
    const unsigned v = sh.best[i];
    r0 += v > v0 || (v == v0 && i < lane);
    r1 += v > v1 || (v == v1 && i < lane + 32);
  }
  const int place = min(K, n - 1);
  const unsigned in0 = __ballot_sync(0xffffffffu, lane < n && r0 == place);
  const unsigned in1 = __ballot_sync(0xffffffffu, lane + 32 < n && r1 == place);
  return value_of(in0 ? __shfl_sync(0xffffffffu, v0, __ffs(in0) - 1) : __shfl_sync(0xffffffffu, v1, __ffs(in1) - 1));
}

// Appends, by all lanes of a warp, the elements k of `hits` to the
// candidates. The order varies from run to run; keys are ranked afterwards.
template <int NT, typename Value>
__device__ __forceinline__ void append(Shared<NT> &sh, unsigned hits, int j0, const Value &value) {
  int total;
  int at = lanes_before<32>(__popc(hits), total);
  if (total == 0) return;
  at += __shfl_sync(0xffffffffu, (threadIdx.x & 31) == 0 ? atomicAdd(&sh.count, total) : 0, 0);
  for (; hits; hits &= hits - 1, ++at) {
    const int k = __ffs(hits) - 1;
    if (at < kCandidates) sh.keys[at] = key_of(value(k), j0 + k);
  }
}

// The part's K first alternatives: put(place, key) by some thread for each.
// top: this thread's maximum over its vectors and single elements; bound from
// join(), which also set the counts to 0.
template <typename T, int NT, typename Put>
__device__ __forceinline__ void alternatives(Shared<NT> &sh, const Part<T> &p, float top, float bound, int K,
                                             const Put &put) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Candidates are what reaches the bound, at least K elements. Where they are
  // too many for the room (ties), or the bound is -inf, only what is above it.
  float low = bound == -INFINITY ? next_up(bound) : bound;
  int above;
  while (true) {
    unsigned slots = 0;
    if (top >= low)
#pragma unroll
      for (int k = 0; k < kSlots<NT>; ++k) slots |= sh.slots[k][tid] >= low ? 1u << k : 0u;
    int total;
    int at = lanes_before<32>(__popc(slots), total);
    if (total) at += __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(&sh.listed, total) : 0, 0);
    for (; slots; slots &= slots - 1) sh.list[at++] = (unsigned short)(tid + NT * (__ffs(slots) - 1));
    if (warp == 0) {  // fewer than 32 single elements
      const bool has = tid < p.singles();
      const int j = has ? p.single(tid) : 0;
      const float v = has ? to_f32(p.x[j]) : -INFINITY;
      append(sh, has && v >= low ? 1u : 0u, j, [&](int) { return v; });
    }
    __syncthreads();
    const int reads = sh.listed * kDeep;
    for (int u0 = 0; u0 * NT < p.vectors; u0 += kSlots<NT> * kDeep)
      for (int i = tid; i - lane < reads; i += NT) {
        int v = p.vectors;
        if (i < reads) {
          const int entry = sh.list[i / kDeep];
          v = vector_of<NT>(u0 + entry / NT * kDeep + i % kDeep, entry % NT);
        }
        const uint4 w = v < p.vectors ? p.load(v) : nothing(T());
        append(sh, reaching<T>(w, low), p.first + v * kVec<T>, [&](int k) { return element<T>(w, k); });
      }
    __syncthreads();
    above = sh.count;
    if (above <= kCandidates || low != bound) break;
    low = next_up(bound);
    __syncthreads();
    if (tid == 0) sh.count = sh.listed = 0;
    __syncthreads();
  }
  if (above > kCandidates) {
    // Rows made so that a few threads hold everything large: one sweep for
    // each alternative.
    Key last = ~0ull;
    for (int k = 0; k < K; ++k) {
      Key best = 0;
      for (int j = p.begin + tid; j < p.end; j += NT) {
        const Key c = key_of(to_f32(p.x[j]), j);
        if (c < last && c > best) best = c;
      }
      best = lanes_max<32>(best);
      __syncthreads();
      if (lane == 0) sh.keys[warp] = best;
      __syncthreads();
      last = sh.keys[0];
      for (int w = 1; w < NT / 32; ++w) last = sh.keys[w] > last ? sh.keys[w] : last;
      if (tid == 0) put(k, last);
    }
    return;
  }
  int n = above;
  if (above < K) {
    // The rest are at the bound (these are above it): the first ones in the
    // row's order, 4 elements a thread and sweep.
    const int need = K - above;
    int found = 0;
    for (int base = p.begin; found < need && base < p.end; base += 4 * NT) {
      const int j0 = base + 4 * tid;
      unsigned hit = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j0 + k < p.end && to_f32(p.x[j0 + k]) == bound) hit |= 1u << k;
      int before = __popc(hit);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += up;
      }
      __syncthreads();  // the last sweep's counts have been read
      if (lane == 31) sh.warp_count[warp] = before;
      __syncthreads();
      int at = found + before - __popc(hit), total = found;
      for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) at += sh.warp_count[w];
        total += sh.warp_count[w];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (hit >> k & 1) {
          if (at < need) sh.keys[above + at] = key_of(bound, j0 + k);
          ++at;
        }
      found = total;
    }
    __syncthreads();
    n = above + min(found, need);
    // a row with NaN in it may leave places open
    if (tid >= n && tid < K) put(tid, key_of(NAN, p.begin + tid));
  }
  // distinct keys: a key's place is the number of larger ones
  for (int c = tid; c < n; c += NT) {
    const Key mine = sh.keys[c];
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += sh.keys[i] > mine;
    if (rank < K) put(rank, mine);
  }
}

// K: whether the alternatives will ask for the slots.
template <typename T, int NT>
__device__ __forceinline__ Running sweep(Shared<NT> &sh, const Part<T> &p, int K) {
  Running r;
  const bool has = (int)threadIdx.x < p.singles();
  const float single = has ? to_f32(p.x[p.single(threadIdx.x)]) : -INFINITY;
  const int whole = p.vectors / (kDeep * NT), groups = (p.vectors + kDeep * NT - 1) / (kDeep * NT);
  const auto load = [&](uint4 (&w)[kDeep], int g) {
    if (g < whole) load_group<NT, true>(w, p, g, threadIdx.x);
    else load_group<NT, false>(w, p, g, threadIdx.x);
  };
  const auto add_group = [&](const uint4 (&w)[kDeep], int g) {
    float each[kDeep];
    const float top = take<T, kDeep>(r, w, each);
    if (K) {
      float &slot = sh.slots[g % kSlots<NT>][threadIdx.x];
      slot = g < kSlots<NT> ? top : fmaxf(top, slot);
    }
  };
  // the next group's vectors are in flight while a group is added; two groups
  // a turn, so that none is copied
  uint4 a[kDeep], b[kDeep];
  load(a, 0);
#pragma unroll 1
  for (int g = 0; g < groups; g += 2) {
    load(b, g + 1);
    add_group(a, g);
    if (g + 1 >= groups) break;
    load(a, g + 2);
    add_group(b, g + 1);
  }
  if (K)
    for (int g = groups; g < kSlots<NT>; ++g) sh.slots[g][threadIdx.x] = -INFINITY;
  if (has) take(r, single);
  return r;
}

// C blocks a row (a cluster where C > 1), part c its c-th share of vectors.
template <typename T, int NT, int C>
__global__ void __launch_bounds__(NT, 1024 / NT)
logprob_fwd_kernel(const T *__restrict__ x, long long stride, Outputs o, long long rows, int V, int K) {
  __shared__ Shared<NT> sh;
  griddep_wait();
  griddep_launch_dependents();
  const int c = C > 1 ? blockIdx.x % C : 0;
  // shares are a multiple of 64 elements; the last one takes what is left
  const int share = C > 1 ? (V / C) & ~63 : V;
  const int begin = c * share, end = c == C - 1 ? V : begin + share;
  for (long long row = blockIdx.x / C; row < rows; row += gridDim.x / C) {
    const T *xr = x + row * stride;
    const Given given(o, xr, row, V, c == 0 && threadIdx.x == 0);
    const Part<T> p(xr, begin, end);
    const Running mine = sweep(sh, p, K);
    float m, s, t;
    const float bound = join(sh, mine, max(1, min(NT < 512 ? NT / 32 : 16, p.vectors / 32)), K, m, s, t);
    if constexpr (C == 1) {
      const Norm norm(m, s);
      if (threadIdx.x == 0) finish(o, row, norm, s, t, given);
      if (K)
        alternatives(sh, p, mine.m, bound, K, [&](int k, Key key) {
          o.top_ids[row * K + k] = index_of(key);
          o.top_logp[row * K + k] = norm.log_p(value_of(key));
        });
      __syncthreads();  // the next row writes what this one has read
    } else {
      if (K) alternatives(sh, p, mine.m, bound, K, [&](int k, Key key) { sh.top[k] = key; });
      if (threadIdx.x == 0) {
        sh.part[0] = m;
        sh.part[1] = s;
        sh.part[2] = t;
      }
      sm103::cluster_sync();
      if (c == 0) {
        // every thread joins the parts in order
        Running all;
        all.m = m;
        all.s = Pair(s, 0.f);
        all.t = Pair(t, 0.f);
        for (int q = 1; q < C; ++q) {
          const uint32_t at = sm103::mapa_shared(sm103::smem_u32(sh.part), q);
          Running b;
          float bs, bt;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(b.m) : "r"(at));
          asm volatile("ld.shared::cluster.f32 %0, [%1+4];" : "=f"(bs) : "r"(at));
          asm volatile("ld.shared::cluster.f32 %0, [%1+8];" : "=f"(bt) : "r"(at));
          b.s = Pair(bs, 0.f);
          b.t = Pair(bt, 0.f);
          if (b.m > all.m) rescale(all, b.m);
          else if (all.m > b.m) rescale(b, all.m);
          all.s = add(all.s, b.s);
          all.t = add(all.t, b.t);
        }
        static_assert(C * kMaxTopK <= kCandidates, "all parts' alternatives fit");
        for (int n = threadIdx.x; n < C * K; n += NT) {
          Key k;
          asm volatile("ld.shared::cluster.u64 %0, [%1];"
                       : "=l"(k)
                       : "r"(sm103::mapa_shared(sm103::smem_u32(&sh.top[n % K]), n / K)));
          sh.keys[n] = k;
        }
        float none;
        all.s.get(s, none);
        all.t.get(t, none);
        const Norm norm(all.m, s);
        if (threadIdx.x == 0) finish(o, row, norm, s, t, given);
        __syncthreads();
        for (int n = threadIdx.x; n < C * K; n += NT) {
          const Key k = sh.keys[n];
          int rank = 0;
          for (int i = 0; i < C * K; ++i) rank += sh.keys[i] > k || (sh.keys[i] == k && i < n);
          if (rank < K) {
            o.top_ids[row * K + rank] = index_of(k);
            o.top_logp[row * K + rank] = norm.log_p(value_of(k));
          }
        }
      }
      sm103::cluster_sync();  // no part is overwritten, or gone, before it was read
    }
  }
}

// ---------------------------------------------------------------- gradient

struct RowGrad {
  float l, a, b, gl;  // dx = p (a + b lp), lp = x - l; gl: the token's own
  int tok;
  bool none;          // all 0, whatever the logits are
};

__device__ __forceinline__ RowGrad row_grad(const int32_t *tokens, const float *lse, const float *entropy,
                                            const float *dlogp, const float *dentropy, long long row, int V) {
  RowGrad g;
  g.l = lse[row];
  g.tok = tokens ? tokens[row] : -1;
  g.gl = g.tok >= 0 && g.tok < V ? dlogp[row] : 0.f;
  const float gh = dentropy ? dentropy[row] : 0.f;
  g.b = -gh;
  g.a = -g.gl - (dentropy ? gh * entropy[row] : 0.f);
  // without a gradient, or nothing but masked logits, of which lse would not
  // tell how many they are
  g.none = (g.gl == 0.f && gh == 0.f) || g.l <= -0x1p24f;
  if (g.l == INFINITY) g.l = NAN;
  return g;
}

__device__ __forceinline__ float grad_of(float v, const RowGrad &g) {
  // clamped where p is 0, so that p lp is 0 there, too (NaN stays)
  const float lp = max_nan(v - g.l, -200.f);
  return ex2(lp * kLog2e) * fmaf(g.b, lp, g.a);
}

template <typename T>
__device__ __forceinline__ void grad_single(const T *x, T *dx, int j, const RowGrad &g) {
  const float v = to_f32(x[j]);
  float d = grad_of(v, g);
  if (j == g.tok && v != -INFINITY) d += g.gl;
  dx[j] = from_f32<T>(g.none ? 0.f : d);
}

// Vector i of a row, held in w.
template <typename T>
__device__ __forceinline__ void grad_vector(T *dr, const Part<T> &p, int i, const uint4 &w, const RowGrad &g) {
  constexpr int W = kVec<T>;
  if (g.none) {
    __stcs((uint4 *)(dr + p.first) + i, make_uint4(0, 0, 0, 0));
    return;
  }
  float v[W], d[W];
  unpack(w, v);
#pragma unroll
  for (int e = 0; e < W; ++e) d[e] = grad_of(v[e], g);
  const int j0 = p.first + i * W;
  if ((unsigned)(g.tok - j0) < (unsigned)W) {
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (j0 + e == g.tok && v[e] != -INFINITY) d[e] += g.gl;
  }
  // not read here again: leaves L2 to the logits (8192 x 50021: 266 -> 248 us)
  __stcs((uint4 *)(dr + p.first) + i, pack(d));
}

constexpr int kThreads = 256;
constexpr int kGradVectors = 4;  // of a thread

// VEC: input and output rows start at the same place of a vector. A block for
// each kGradVectors kThreads vectors of a row (half and twice as many: 274 and
// 284 us at 8192 x 50021, 247 so). dx may be x.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) logprob_bwd_kernel(const T *x, long long stride, const int32_t *tokens,
                                                               const float *lse, const float *entropy,
                                                               const float *dlogp, const float *dentropy, T *dx,
                                                               long long dstride, long long rows, int V, int pieces) {
  griddep_wait();
  griddep_launch_dependents();
  const long long work = rows * pieces;
  for (long long b = blockIdx.x; b < work; b += gridDim.x) {
    const long long row = b / pieces;
    const int piece = (int)(b - row * pieces);
    const T *xr = x + row * stride;
    T *dr = dx + row * dstride;
    if constexpr (VEC) {
      const Part<T> p(xr, 0, V);
      uint4 w[kGradVectors];
      const int v0 = piece * kGradVectors * kThreads + threadIdx.x;
#pragma unroll
      for (int k = 0; k < kGradVectors; ++k)
        if (v0 + k * kThreads < p.vectors) w[k] = p.load(v0 + k * kThreads);
      const RowGrad g = row_grad(tokens, lse, entropy, dlogp, dentropy, row, V);
#pragma unroll
      for (int k = 0; k < kGradVectors; ++k) {
        const int i = v0 + k * kThreads;
        if (i < p.vectors) grad_vector(dr, p, i, w[k], g);
      }
      if (piece == 0 && (int)threadIdx.x < p.singles()) grad_single(xr, dr, p.single(threadIdx.x), g);
    } else {
      const RowGrad g = row_grad(tokens, lse, entropy, dlogp, dentropy, row, V);
      const int j0 = piece * kGradVectors * kThreads * kVec<T>;
      const int j1 = min(V, j0 + kGradVectors * kThreads * kVec<T>);
#pragma unroll 4
      for (int j = j0 + threadIdx.x; j < j1; j += kThreads) grad_single(xr, dr, j, g);
    }
  }
}

constexpr int kShort = 1024;  // longest row of a few lanes

// Short rows: 8 lanes a row where rows go by vectors, else a warp.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) logprob_bwd_short_kernel(const T *x, long long stride, const int32_t *tokens,
                                                                     const float *lse, const float *entropy,
                                                                     const float *dlogp, const float *dentropy, T *dx,
                                                                     long long dstride, long long rows, int V) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int L = VEC ? 8 : 32, per = kThreads / L;
  const int lane = (int)threadIdx.x % L;
  for (long long row = (long long)blockIdx.x * per + threadIdx.x / L; row < rows; row += (long long)gridDim.x * per) {
    const T *xr = x + row * stride;
    T *dr = dx + row * dstride;
    if constexpr (VEC) {
      const Part<T> p(xr, 0, V);
      uint4 w[kGradVectors];
#pragma unroll
      for (int k = 0; k < kGradVectors; ++k)
        if (k * L + lane < p.vectors) w[k] = p.load(k * L + lane);
      const RowGrad g = row_grad(tokens, lse, entropy, dlogp, dentropy, row, V);
      for (int base = 0; base < p.vectors; base += kGradVectors * L) {
#pragma unroll
        for (int k = 0; k < kGradVectors; ++k)
          if (base + k * L + lane < p.vectors) grad_vector(dr, p, base + k * L + lane, w[k], g);
#pragma unroll
        for (int k = 0; k < kGradVectors; ++k) {
          const int i = base + (kGradVectors + k) * L + lane;
          if (i < p.vectors) w[k] = p.load(i);
        }
      }
      for (int s = lane; s < p.singles(); s += L) grad_single(xr, dr, p.single(s), g);
    } else {
      const RowGrad g = row_grad(tokens, lse, entropy, dlogp, dentropy, row, V);
#pragma unroll 4
      for (int j = lane; j < V; j += L) grad_single(xr, dr, j, g);
    }
  }
}

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

unsigned grid_of(long long blocks) { return (unsigned)(blocks < (1LL << 30) ? blocks : (1LL << 30)); }

template <typename T, int L>
cudaError_t launch_short(const LogprobArgs &a, const T *x, long long stride, const Outputs &o, cudaStream_t st) {
  // Resident blocks that take rows in turn; with alternatives in bf16, whose
  // rows take longer than their loads and not equally long, four times as many
  // (us: 20000 x 1000, 5 alternatives, 18.6 against 20.4; 5000 x 8000, 8, 23.8
  // and 26.6; without alternatives 12.6 and 12.1; f32 20000 x 4000, 5, 66 and 65).
  const long long per = kShortThreads / L, blocks = (a.rows + per - 1) / per;
  const long long most = (long long)short_blocks(a.top_k) * sm_count() * (a.top_k && sizeof(T) == 2 ? 4 : 1);
  const auto k = a.top_k ? logprob_short_kernel<T, L, true> : logprob_short_kernel<T, L, false>;
  return launch_ex(k, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kShortThreads), 0,
                   st, 1, x, stride, o, a.rows, a.V, a.top_k);
}

template <typename T, int NT, int C>
cudaError_t launch_long(const LogprobArgs &a, const T *x, long long stride, const Outputs &o, cudaStream_t st) {
  const long long rows = a.rows < (1LL << 26) ? a.rows : (1LL << 26);
  return launch_ex(logprob_fwd_kernel<T, NT, C>, dim3((unsigned)(rows * C)), dim3(NT), 0, st, C, x, stride, o, a.rows,
                   a.V, a.top_k);
}

template <typename T>
cudaError_t fwd(const LogprobArgs &a, const T *x, long long stride, const Outputs &o, cudaStream_t st) {
  const int vectors = a.V / kVec<T>;
  const long long sms = sm_count();
  // More rows than 128-thread blocks fit at once: rows up to 1280 vectors go
  // to a warp or less, without barriers (1500 x 2000 bf16, 8 alternatives: 6.3
  // against 10.9 us with such a block a row; 600 x 2000: 6.3 against 5.9).
  const bool many = a.rows > 8 * sms;
  // Lanes a row: what a row costs besides its elements is shared by a warp's
  // rows, as long as K + 1 of two maxima a lane leave few candidates and a
  // lane's vectors are few (20000 rows, us with 8, 16 and 32 lanes: 256 f32, 8
  // alternatives 14.3, 17.6, -; 20 alternatives -, 24, 37; 2000 bf16, 10
  // alternatives 37, 31, -; 8000 bf16, 5 alternatives -, 78, 71).
  if (vectors <= 128 && a.top_k <= 10) return launch_short<T, 8>(a, x, stride, o, st);
  if (vectors <= (many ? 512 : 128) && a.top_k <= 28) return launch_short<T, 16>(a, x, stride, o, st);
  if (a.V <= 1024 || (vectors <= 1280 && many)) return launch_short<T, 32>(a, x, stride, o, st);
  // A few very long rows: a cluster of 8 blocks each, on SMs of their own (1 x
  // 262144 f32, 8 alternatives: 9.5 us against 18 with 1024 threads; its
  // barriers cost 3 us, so 20 x 50021 bf16 takes 8.5 us against 7.7), or of 4
  // or 2 larger ones (32 x 262144 bf16 9.6 us, one block 15.8; 64 x 131072 9.3
  // and 10.2; 70 x 100000 9.3 and 9.7; 70 x 65536 8.0 and 7.7).
  if (a.V >= 65536 && a.rows * 8 <= sms) return launch_long<T, 256, 8>(a, x, stride, o, st);
  if (a.V >= 98304 && a.rows * 4 <= sms) return launch_long<T, 512, 4>(a, x, stride, o, st);
  if (a.V >= 98304 && a.rows * 2 <= sms) return launch_long<T, 512, 2>(a, x, stride, o, st);
  // Many rows of middling length: 64-thread blocks, whose barriers wait for
  // two warps only (5 alternatives, bf16: 8192 x 16000 57 us, 67 with 128, 60
  // with a warp a row; 20000 x 10000 97, 136 and 87; 8192 x 50021 143 and 146,
  // but with 20 alternatives 160 and 155).
  if (a.rows > 4 * sms && vectors <= 5000) return launch_long<T, 64, 1>(a, x, stride, o, st);
  // Threads a row: 1024 on every SM, while each has 15 vectors or more (300 x
  // 131072 bf16: 19.5 us with 512, 20.4 with 256, 27 with 128; 300 x 50021:
  // 12.4, 11.1 and 13.2). With more rows the rows in flight fill L2 from
  // 128-thread blocks of very long rows (2000 x 262144: 193 us, 183 with 256;
  // 8192 x 50021: 151 us, 178 with 256).
  if (a.rows <= 2 * sms && vectors >= 15 * 512) return launch_long<T, 512, 1>(a, x, stride, o, st);
  if ((a.rows <= 4 * sms && vectors >= 15 * 256) || vectors > 16384) return launch_long<T, 256, 1>(a, x, stride, o, st);
  return launch_long<T, 128, 1>(a, x, stride, o, st);
}

template <typename T>
cudaError_t bwd(const LogprobArgs &a, const T *x, long long stride, const int32_t *tokens, const float *lse,
                const float *entropy, const float *dlogp, const float *dentropy, T *dx, long long dstride,
                cudaStream_t st) {
  // input and output rows start at the same place of a vector
  const bool vec = (uintptr_t)x % 16 == (uintptr_t)dx % 16 && (a.rows == 1 || (stride - dstride) % kVec<T> == 0);
  if (a.V <= kShort) {
    const int rows = vec ? kThreads / 8 : kThreads / 32;  // of a block
    return launch_ex(vec ? logprob_bwd_short_kernel<T, true> : logprob_bwd_short_kernel<T, false>,
                     dim3(grid_of((a.rows + rows - 1) / rows)), dim3(kThreads), 0, st, 1, x, stride, tokens, lse,
                     entropy, dlogp, dentropy, dx, dstride, a.rows, a.V);
  }
  const int per = kGradVectors * kThreads * kVec<T>;
  const int pieces = (a.V + per - 1) / per;
  const long long blocks = a.rows < (1LL << 30) / pieces ? a.rows * pieces : 1LL << 30;
  return launch_ex(vec ? logprob_bwd_kernel<T, true> : logprob_bwd_kernel<T, false>, dim3(grid_of(blocks)),
                   dim3(kThreads), 0, st, 1, x, stride, tokens, lse, entropy, dlogp, dentropy, dx, dstride, a.rows, a.V,
                   pieces);
}

}  // namespace

cudaError_t launch_logprob_fwd(const LogprobArgs &a, const void *x, long long stride, const int32_t *tokens,
                               float *logp, float *lse, float *entropy, int32_t *top_ids, float *top_logp,
                               cudaStream_t st, int *launches) {
  const Outputs o = {tokens, logp, lse, entropy, top_ids, top_logp};
  const cudaError_t e = a.dtype == RXL_DTYPE_BF16 ? fwd(a, (const __nv_bfloat16 *)x, stride, o, st)
                                                  : fwd(a, (const float *)x, stride, o, st);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_logprob_bwd(const LogprobArgs &a, const void *x, long long stride, const int32_t *tokens,
                               const float *lse, const float *entropy, const float *dlogp, const float *dentropy,
                               void *dx, long long dx_stride, cudaStream_t st, int *launches) {
  const cudaError_t e =
      a.dtype == RXL_DTYPE_BF16
          ? bwd(a, (const __nv_bfloat16 *)x, stride, tokens, lse, entropy, dlogp, dentropy, (__nv_bfloat16 *)dx,
                dx_stride, st)
          : bwd(a, (const float *)x, stride, tokens, lse, entropy, dlogp, dentropy, (float *)dx, dx_stride, st);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaGetLastError();
}

}  // namespace rxl
