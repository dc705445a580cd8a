// LayerNorm with an optional residual sum, and its backward with the
// reduction of the weights' gradients (include/rxl.h: rxl_layernorm_*).
//
// Memory-bound: a row is read once, held in registers, and written once. A
// group of G threads takes a row, E elements a thread, so the sweeps over the
// row that the statistics take (sum, then squared differences; two more where
// the mean is far larger than the spread) and the output run on registers; a
// group is a few lanes or a warp (shuffles) or several warps (a named barrier
// around a few words of shared memory). Groups are mostly persistent: they keep
// their columns of gamma and beta, and the next row's loads are in flight while
// a row is worked on.
//
// The backward keeps, for its columns, running sums of dy xh and dy over its
// rows: dgamma and dbeta cost no second reading of dy and s. A block joins
// its groups' sums in shared memory and writes one partial row; a second
// kernel adds the partial rows in block order, so results do not depend on
// timing (of few rows one block writes the result). The sums leave few
// registers, so rows come by asynchronous copies into each thread's own words
// of shared memory, three rows deep, and are read from there for both sweeps.
//
// Measured (the card copies at 6.78 TB/s): forward with residual, bf16, 8192 x
// 1024 12.2 us (5.5 TB/s: five turns of 1824 rows, the last half empty), 32768 x
// 4096 163 us (6.6), without one 30000 x 4096 78 us (6.3); backward bf16 65536 x
// 1024 62 us (6.5), 32768 x 4096 135 us (6.0), 8192 x 1024 13.4 us (3.8), f32
// 5001 x 1023 14.9 us (4.1). What bounds the backward: 7 to 10 us for the first
// rows, the partial sums and the second launch; beyond that 16 warps on an SM
// (its sums), a row's two sweeps one after the other, within 10% of memory.
#include <math.h>

#include "sm103.cuh"
#include "stream_common.cuh"
#include "train.cuh"

namespace rxl {
namespace {

using namespace stream;
using sm103::griddep_launch_dependents;
using sm103::griddep_wait;

// Threads resident on an SM in the backward: its sums take 2 E registers each.
// (E 16: 65536 x 1024 bf16 68 us with 512, 77 with 768 and spills; E 8: 20000 x
// 1024 f32 41 us with 768, 43 with 512; E 32: see by_width_bf16.)
constexpr int bwd_threads(int E) { return E <= 8 ? 768 : E <= 24 ? 512 : 384; }
// Rows of a thread in flight or in hand (2, 3, 4 and 6, bf16 us: 8192 x 1024
// 13.4, 13.4, 14.0 and 15.3; 32768 x 4096 141, 135, 136 and 138; 2048 x 4096
// 16.9, 16.5, 17.2 and 18.8. The next row in registers instead, with 16
// elements a thread: 72 against 68 us at 65536 x 1024).
constexpr int kStages = 3;

// A group's place in its block and the E elements its threads hold. VEC:
// whole 16-byte vectors, vector i of thread t at (i G + t); else single
// elements, element i of thread t at i G + t (rows that do not all start on
// 16 bytes). Arithmetic is on pairs of elements.
template <typename T, int G, int E, bool VEC>
struct Row {
  static constexpr int kThreads = G > 256 || 256 % G ? G : E <= 24 || G > 128 ? 256 : 128;  // of a block
  static constexpr int kGroups = kThreads / G;
  static constexpr int kWarps = G > 32 ? G / 32 : 1;
  static constexpr int kW = VEC ? kVec<T> : 1;  // consecutive elements
  static constexpr int kN = E / kW;             // pieces a thread
  static constexpr int kP = E / 2;              // pairs a thread
  [[maybe_unused]] static constexpr int kE = E;

  static __device__ __forceinline__ int lane() { return (int)threadIdx.x % G; }
  static __device__ __forceinline__ int column(int i) { return (i * G + lane()) * kW; }
  static __device__ __forceinline__ int column_of(int e, int t) { return (e / kW * G + t) * kW + e % kW; }

  // What a thread holds of a row as it is stored; elements beyond the row
  // are 0 (D == 0: no row at all).
  struct Raw {
    uint4 v[VEC ? kN : 1];
    T e[VEC ? 1 : E];
  };
  static __device__ __forceinline__ void read(Raw &r, const T *row, int D) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = column(i);
      if constexpr (VEC) r.v[i] = c < D ? *(const uint4 *)(row + c) : make_uint4(0, 0, 0, 0);
      else r.e[i] = c < D ? row[c] : from_f32<T>(0.f);
    }
  }
  // Pair p of the thread's elements.
  static __device__ __forceinline__ Pair pair(const Raw &r, int p) {
    if constexpr (!VEC) {
      return Pair(to_f32(r.e[2 * p]), to_f32(r.e[2 * p + 1]));
    } else if constexpr (sizeof(T) == 2) {
      const uint4 &w = r.v[p / 4];
      const uint32_t u = p % 4 == 0 ? w.x : p % 4 == 1 ? w.y : p % 4 == 2 ? w.z : w.w;
      return Pair(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    } else {
      const uint4 &w = r.v[p / 2];
      return p % 2 == 0 ? Pair(__uint_as_float(w.x), __uint_as_float(w.y))
                        : Pair(__uint_as_float(w.z), __uint_as_float(w.w));
    }
  }
  // Writes piece i from the thread's pairs.
  static __device__ __forceinline__ void write(T *row, int D, int i, const Pair (&v)[kP]) {
    const int c = column(i);
    if (c >= D) return;
    if constexpr (VEC) {
      float f[kW];
#pragma unroll
      for (int k = 0; k < kW / 2; ++k) v[i * kW / 2 + k].get(f[2 * k], f[2 * k + 1]);
      *(uint4 *)(row + c) = pack(f);
    } else {
      float f[2];
      v[i / 2].get(f[0], f[1]);
      row[c] = from_f32<T>(f[i % 2]);
    }
  }
  // The same pairs, 0 where they lie beyond the row.
  static __device__ __forceinline__ Pair inside(Pair v, int p, int D) {
    float a, b;
    v.get(a, b);
    return Pair(column(2 * p / kW) < D ? a : 0.f, column((2 * p + 1) / kW) < D ? b : 0.f);
  }
  // Keeps the compiler from holding on to floats that were unpacked before.
  static __device__ __forceinline__ void renew(Raw &r) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if constexpr (VEC) asm volatile("" : "+r"(r.v[i].x), "+r"(r.v[i].y), "+r"(r.v[i].z), "+r"(r.v[i].w));
      else if constexpr (sizeof(T) == 2) asm volatile("" : "+h"(*(unsigned short *)&r.e[i]));
      else asm volatile("" : "+f"(*(float *)&r.e[i]));
    }
  }

  // A row's pieces copied to this thread's own words of shared memory and
  // read back by it alone: the copies need no registers and no barrier.
  // (Single elements gain nothing: four bytes a copy.)
  [[maybe_unused]] static constexpr bool kStaged = VEC;
  static constexpr int kBytes = E * (int)sizeof(T);  // of a thread
  static __device__ __forceinline__ uint32_t slot(uint32_t base, int i) {
    return base + (i * kThreads + threadIdx.x) * 16;
  }
  static __device__ __forceinline__ void copy(uint32_t base, const T *row, int D) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int c = column(i);
      const bool in = c < D;  // else zeros, and nothing is read
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot(base, i)), "l"(in ? row + c : row),
                   "r"(in ? 16 : 0)
                   : "memory");
    }
  }
  static __device__ __forceinline__ void read_copy(Raw &r, uint32_t base) {
#pragma unroll
    for (int i = 0; i < (VEC ? kN : 0); ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.v[i].x), "=r"(r.v[i].y), "=r"(r.v[i].z), "=r"(r.v[i].w)
                   : "r"(slot(base, i))
                   : "memory");
  }

  // Sums of NV values over the group, the same in every thread. `slot` flips
  // between two sets of words, so one barrier a sum is enough: a warp writes
  // a set again only after the next sum's barrier, which every warp reaches
  // after it has read the set.
  template <int NV>
  static __device__ __forceinline__ void sum(float (&v)[NV], float (*shared)[kGroups][NV][kWarps], int &slot) {
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < NV; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (kWarps > 1) {
      const int g = (int)threadIdx.x / G, w = lane() / 32;
      float(*s)[kWarps] = shared[slot][g];
      slot ^= 1;
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < NV; ++k) s[k][w] = v[k];
      asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(G) : "memory");
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < kWarps; ++j) a += s[k][j];
        v[k] = a;
      }
    }
  }
};

__device__ __forceinline__ float both(Pair p) {
  float a, b;
  p.get(a, b);
  return a + b;
}

// The next row is in flight while a thread's part of it leaves registers for
// that: 64 bytes on 512 threads an SM, with a residual 32 on 768. Wider parts
// are read when their turn comes, and gamma and beta each time; a group for
// every row makes up for it (9000 x 16384 bf16 with residual: 170 us; two
// persistent blocks an SM 199, one 231; 40000 x 1536: 72, ahead 84; without
// residual 45, ahead 43; 20000 x 5120 84 and 75).
template <typename R, bool RES>
constexpr bool can_ahead() { return R::kBytes <= (RES || !R::kStaged ? 32 : 64); }
template <typename R, bool AHEAD>
constexpr int fwd_blocks() { return (!AHEAD ? 1024 : R::kBytes > 32 ? 512 : 768) / R::kThreads; }

// A block's groups take rows in turn. A warp that holds several rows goes on
// while its first one exists (shuffles need every lane); a lane whose own
// row does not reads nothing, writes nothing and adds 0.

// x, residual, y and sum may be the same rows: no __restrict__.
template <typename T, int G, int E, bool VEC, bool RES, bool AHEAD>
__global__ void __launch_bounds__(Row<T, G, E, VEC>::kThreads, fwd_blocks<Row<T, G, E, VEC>, AHEAD>())
norm_fwd_kernel(const T *x, long long xs, const T *res, long long rs, const T *gamma, const T *beta, T *y,
                long long ys, T *sum, long long ss, float *mean, float *rstd, long long rows, int width, float eps) {
  using R = Row<T, G, E, VEC>;
  __shared__ float shared[2][R::kGroups][1][R::kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const long long step = (long long)gridDim.x * R::kGroups;
  long long row = (long long)blockIdx.x * R::kGroups + threadIdx.x / G;
  long long first = (long long)blockIdx.x * R::kGroups + (threadIdx.x & ~31) / G;  // the warp's
  if (first >= rows) return;
  typename R::Raw xn, rn, gm, bt;
  if (AHEAD) {
    const int D = row < rows ? width : 0;
    R::read(xn, x + row * xs, D);
    if (RES) R::read(rn, res + row * rs, D);
    R::read(gm, gamma, width);
    R::read(bt, beta, width);
  }
  const float inv_d = 1.f / width;
  int slot = 0;
#pragma unroll 1
  for (; first < rows; first += step, row += step) {
    const int D = row < rows ? width : 0;
    if (!AHEAD) {
      R::read(xn, x + row * xs, D);
      if (RES) R::read(rn, res + row * rs, D);
    }
    Pair s[R::kP], acc(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < R::kP; ++p) {
      s[p] = R::pair(xn, p);
      if (RES) {
        s[p] = add(s[p], R::pair(rn, p));
        if constexpr (sizeof(T) == 2) {  // the sum is what is stored: rounded to the rows' type
          float a, b;
          s[p].get(a, b);
          const uint32_t u = pack2(a, b);
          s[p] = Pair(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
        }
      }
      acc = add(acc, s[p]);
    }
    if (AHEAD && first + step < rows) {
      const int next = row + step < rows ? width : 0;
      R::read(xn, x + (row + step) * xs, next);
      if (RES) R::read(rn, res + (row + step) * rs, next);
    }
    float a[1] = {both(acc)};
    R::sum(a, shared, slot);
    float mu = a[0] * inv_d;
    if (RES && sum)
#pragma unroll
      for (int i = 0; i < R::kN; ++i) R::write(sum + row * ss, D, i, s);
    // Takes `off` from the row; a[0]: the sum of the squares that are left.
    const auto centre = [&](float off) {
      acc = Pair(0.f, 0.f);
      const Pair neg(-off, -off);
#pragma unroll
      for (int p = 0; p < R::kP; ++p) {
        s[p] = R::inside(add(s[p], neg), p, width);
        acc = fma(s[p], s[p], acc);
      }
      a[0] = both(acc);
      R::sum(a, shared, slot);
    };
    // What rounding left of the mean is the differences' own mean. It counts
    // only where the mean is far larger than the spread (1000.1 everywhere: y
    // off by 0.02): such rows are centred once more. A warp's other rows by 0.
    const auto far = [&]() { return mu * mu > 256.f * (a[0] * inv_d + eps); };
    const auto any_far = [&]() { return G < 32 ? __any_sync(0xffffffffu, far()) : far(); };
    const auto rest = [&]() {
      acc = Pair(0.f, 0.f);
#pragma unroll
      for (int p = 0; p < R::kP; ++p) acc = add(acc, s[p]);
      float r[1] = {both(acc)};
      R::sum(r, shared, slot);
      return far() ? r[0] * inv_d : 0.f;
    };
    // How the rare case is written decides what the usual one costs, whose
    // registers are few (us without it, with it as a loop, and as a branch that
    // centres again or that takes D c^2 from the squares: with residual 32768 x
    // 4096 bf16 162, 162, 166, 166; without 65536 x 1024 42.4, 44.6, 43.6, 42.8;
    // 32768 x 4096 85.0, 86.7, 85.7, 88.8; 4500 x 16384 f32 94, 95, 102, 105).
    // Where all rows are far (mean 100, spread 1): 32768 x 4096 177 and 90 us,
    // 65536 x 1024 without residual 43.2.
    if constexpr (RES || !AHEAD) {
      float off = mu;
#pragma unroll 1
      for (bool first_time = true;; first_time = false) {
        centre(off);
        if (!first_time || !any_far()) break;
        off = rest();
        mu += off;
      }
    } else {
      centre(mu);
      if (any_far()) {
        const float c = rest();
        mu += c;
        if constexpr (G > 32) {
          centre(c);
        } else {
          a[0] = max_nan(fmaf(-c * width, c, a[0]), 0.f);
#pragma unroll
          for (int p = 0; p < R::kP; ++p) s[p] = add(s[p], Pair(-c, -c));
        }
      }
    }
    const float inv = 1.f / sqrtf(a[0] * inv_d + eps);
    if (!AHEAD) {
      R::read(gm, gamma, width);
      R::read(bt, beta, width);
    }
    const Pair scale(inv, inv);
#pragma unroll
    for (int p = 0; p < R::kP; ++p) s[p] = fma(mul(s[p], scale), R::pair(gm, p), R::pair(bt, p));
#pragma unroll
    for (int i = 0; i < R::kN; ++i) R::write(y + row * ys, D, i, s);
    if (mean && R::lane() == 0 && row < rows) {
      mean[row] = mu;
      rstd[row] = inv;
    }
  }
}

template <typename R>
constexpr int bwd_blocks() {  // on an SM
  return bwd_threads(R::kE) > R::kThreads ? bwd_threads(R::kE) / R::kThreads : 1;
}
// Rows of dy and s that a thread has in flight or in hand.
template <typename R>
constexpr int bwd_stages() {
  if (!R::kStaged) return 0;
  constexpr int resident = bwd_blocks<R>() * R::kThreads;
  // a block of the widest rows spills, and the spills need some L1 (9000 x
  // 16384 bf16: 163 us with two stages, 207 with three)
  constexpr int room = (R::kE * R::kThreads > 8192 ? 131072 : 196608) / (resident * 2 * R::kBytes);
  return room > kStages ? kStages : room;
}
template <typename R>
constexpr int bwd_shared() {  // bytes: the stages; at the end the groups' sums
  constexpr int stages = bwd_stages<R>() * 2 * R::kBytes * R::kThreads, sums = R::kGroups > 1 ? R::kP * 16 * R::kThreads : 0;
  return stages > sums ? stages : sums;
}

__device__ __forceinline__ void store(float *p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void store(float *p, const float (&v)[4]) { *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]); }

// pg, pb: block i's sums of dy xh and dy over its rows go to pg + i stride and
// pb + i stride. dx may be the rows of dy or s: no __restrict__.
template <typename T, int G, int E, bool VEC>
__global__ void __launch_bounds__(Row<T, G, E, VEC>::kThreads, bwd_blocks<Row<T, G, E, VEC>>())
norm_bwd_kernel(const T *dy, long long ys, const T *s, long long ss, const T *gamma, const float *mean,
                const float *rstd, T *dx, long long xs, float *pg, float *pb, int stride, long long rows, int width) {
  using R = Row<T, G, E, VEC>;
  constexpr int S = bwd_stages<R>();
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ float shared[2][R::kGroups][2][R::kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const long long step = (long long)gridDim.x * R::kGroups;
  long long row = (long long)blockIdx.x * R::kGroups + threadIdx.x / G;
  long long first = (long long)blockIdx.x * R::kGroups + (threadIdx.x & ~31) / G;  // the warp's
  Pair dg[R::kP], db[R::kP];
#pragma unroll
  for (int p = 0; p < R::kP; ++p) dg[p] = db[p] = Pair(0.f, 0.f);
  const uint32_t base = sm103::smem_u32(dynamic);
  const auto at = [&](int stage, int which) { return base + (stage * 2 + which) * (R::kBytes * R::kThreads); };
  const auto fetch = [&](int stage, long long r) {
    const bool in = r < rows;
    R::copy(at(stage, 0), dy + (in ? r : 0) * ys, in ? width : 0);
    R::copy(at(stage, 1), s + (in ? r : 0) * ss, in ? width : 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (first < rows) {
    typename R::Raw yc, sc, gm;
    if (S > 0)
#pragma unroll
      for (int k = 0; k + 1 < S; ++k) fetch(k, row + k * step);
    const bool live = row < rows;
    float mn = live ? mean[row] : 0.f, in = live ? rstd[row] : 0.f;
    constexpr bool keep_gamma = E * sizeof(T) <= 64;
    if (keep_gamma) R::read(gm, gamma, width);
    const float inv_d = 1.f / width;
    int slot = 0, stage = 0;
#pragma unroll 1
    for (; first < rows; first += step, row += step) {
      const int D = row < rows ? width : 0;
      const float mu = mn, inv = in;
      // this row's copies have landed; the stage freed by the last row takes
      // the one S - 1 rows on
      if constexpr (S == 1) fetch(0, row);
      if constexpr (S > 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S > 1 ? S - 2 : 0) : "memory");
        fetch(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * step);
      } else if constexpr (S == 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      const auto load = [&]() {
        if constexpr (S > 0) {
          R::read_copy(yc, at(stage, 0));
          R::read_copy(sc, at(stage, 1));
        } else {
          R::read(yc, dy + row * ys, D);
          R::read(sc, s + row * ss, D);
        }
        if (!keep_gamma) R::read(gm, gamma, width);
      };
      load();
      if (first + step < rows) {
        const bool next = row + step < rows;
        mn = next ? mean[row + step] : 0.f;
        in = next ? rstd[row + step] : 0.f;
      }
      const Pair neg(-mu, -mu), scale(inv, inv);
      Pair c0(0.f, 0.f), c1(0.f, 0.f);
#pragma unroll
      for (int p = 0; p < R::kP; ++p) {
        // beyond the row dy is 0, and so is what it adds
        const Pair g = R::pair(yc, p), z = mul(add(R::pair(sc, p), neg), scale);
        dg[p] = fma(g, z, dg[p]);
        db[p] = add(db[p], g);
        const Pair h = mul(g, R::pair(gm, p));
        c0 = add(c0, h);
        c1 = fma(h, z, c1);
      }
      float c[2] = {both(c0), both(c1)};
      R::sum(c, shared, slot);
      // the row once more, instead of holding on to its floats
      if (S > 0 || !keep_gamma) {
        load();
      } else {
        R::renew(yc);
        R::renew(sc);
      }
      // rstd (g - mean(g) - xh mean(g xh)) as g rstd + ((s - mu) k + a)
      const float a = -c[0] * inv_d * inv, k = -c[1] * inv_d * inv * inv;
      const Pair pa(a, a), pk(k, k);
      Pair d[R::kP];
#pragma unroll
      for (int p = 0; p < R::kP; ++p)
        d[p] = fma(mul(R::pair(yc, p), R::pair(gm, p)), scale, fma(add(R::pair(sc, p), neg), pk, pa));
#pragma unroll
      for (int i = 0; i < R::kN; ++i) R::write(dx + row * xs, D, i, d);
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  // Whole sectors: four columns a store where a thread's columns are
  // consecutive (2048 x 4096 bf16: 17 us, 24 with single ones).
  float *const og = pg + (size_t)blockIdx.x * stride, *const ob = pb + (size_t)blockIdx.x * stride;
  constexpr int kQ = VEC ? 4 : 1;
  if constexpr (R::kGroups > 1) {  // the groups' sums of each column, in group order
    float *joined = (float *)dynamic;
    __syncthreads();  // every thread is done with its stages
#pragma unroll
    for (int p = 0; p < R::kP; ++p) {
      dg[p].get(joined[(2 * p) * R::kThreads + threadIdx.x], joined[(2 * p + 1) * R::kThreads + threadIdx.x]);
      db[p].get(joined[(E + 2 * p) * R::kThreads + threadIdx.x], joined[(E + 2 * p + 1) * R::kThreads + threadIdx.x]);
    }
    __syncthreads();
    constexpr int kPer = R::kW / kQ;  // stores of a piece
    for (int i = threadIdx.x; i < 2 * E * G / kQ; i += R::kThreads) {
      const int t = i / kPer % G, piece = i / (kPer * G);  // of both sums' pieces
      const int e = piece * R::kW + i % kPer * kQ, c = R::column_of(e % E, t);
      if (c < width) {
        float a[kQ];
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
          a[q] = 0.f;
#pragma unroll 4
          for (int g = 0; g < R::kGroups; ++g) a[q] += joined[(e + q) * R::kThreads + g * G + t];
        }
        store((e < E ? og : ob) + c, a);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; e += kQ) {
      const int c = R::column_of(e, R::lane());
      float g[E], b[E];
#pragma unroll
      for (int p = 0; p < R::kP; ++p) {
        dg[p].get(g[2 * p], g[2 * p + 1]);
        db[p].get(b[2 * p], b[2 * p + 1]);
      }
      if (c < width) {
        float a[kQ];
#pragma unroll
        for (int q = 0; q < kQ; ++q) a[q] = g[e + q];
        store(og + c, a);
#pragma unroll
        for (int q = 0; q < kQ; ++q) a[q] = b[e + q];
        store(ob + c, a);
      }
    }
  }
}

// Column sums of part [P][2 D] in a fixed order, C columns a block. What
// bounds it is one wait after the other: with 8 columns a thread has 5 rows'
// values in flight, all it has of up to 320 partial rows (of 456, three blocks
// an SM, it has 8, in two turns); with 32 there are fewer blocks to start, which
// is better for few rows or wide ones (backward of 8192 x 1024 bf16 with 8 and
// 32 columns 13.6 and 14.5 us, 2048 x 1024 6.6 and 8.1, 512 x 1024 4.3 and 4.0,
// 2048 x 8192 27.9 and 26.0).
constexpr int kJoinThreads = 512;
template <int C>
__global__ void __launch_bounds__(kJoinThreads) norm_bwd_join_kernel(const float *part, float *dgamma, float *dbeta,
                                                                     int P, int D) {
  constexpr int kSlices = kJoinThreads / C, kWarps = kJoinThreads / 32;
  constexpr int kAtOnce = C == 8 ? 5 : 1, kUnroll = C == 8 ? 1 : 8;
  __shared__ float s[kWarps][C];
  griddep_wait();
  griddep_launch_dependents();
  const int col = threadIdx.x % C, c = blockIdx.x * C + col;
  float a = 0.f;
  if (c < 2 * D) {
#pragma unroll kUnroll
    for (int p = threadIdx.x / C; p < P; p += kSlices * kAtOnce) {
      float v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        v[k] = k == 0 || p + k * kSlices < P ? part[(size_t)(p + k * kSlices) * 2 * D + c] : 0.f;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) a += v[k];
    }
  }
#pragma unroll
  for (int o = C; o < 32; o *= 2) a += __shfl_xor_sync(0xffffffffu, a, o);
  if ((threadIdx.x & 31) < C) s[threadIdx.x / 32][col] = a;
  __syncthreads();
  if (threadIdx.x < C && c < 2 * D) {
#pragma unroll
    for (int k = 1; k < kWarps; ++k) a += s[k][col];
    if (c < D) dgamma[c] = a;
    else dbeta[c - D] = a;
  }
}

constexpr int kMaxPartials = 456;  // blocks of the backward: three on each of 152 SMs

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Lets a kernel (one per template instance) take `bytes` of shared memory, once for each device.
template <typename... A>
cudaError_t allow_shared_on(void (*k)(A...), int bytes, std::atomic<unsigned long long> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <bool RES>
struct Fwd {
  static constexpr bool kBackward = false, kResidual = RES;
  NormArgs a;
  const void *x, *res, *gamma, *beta;
  void *y, *sum;
  long long xs, rs, ys, ss;
  float *mean, *rstd;
  cudaStream_t st;

  template <typename T, int G, int E, bool VEC>
  cudaError_t run() const {
    using R = Row<T, G, E, VEC>;
    // Groups that hold everything the next row needs are persistent. With a
    // residual, which doubles what is in flight, a group for every row is
    // faster in bf16 where the rows are many, or all fit at once, and leave few
    // lanes idle (us, persistent and not: 65536 x 1024 90 and 83, 30000 x 2000
    // 77 and 76, 30000 x 1800 66 and 72, 32768 x 4096 170 and 163, 4096 x 4096
    // 22 and 23, 9000 x 8192 96 and 103, 2048 x 1024 3.6 and 3.2; blocks of
    // 160, 30000 x 2560, 92 and 113).
    if constexpr (can_ahead<R, RES>()) {
      if constexpr (RES && sizeof(T) == 2 && VEC && 256 % G == 0)
        if (a.D * 16 >= G * E * 15 &&
            (a.rows <= (long long)sm_count() * (1024 / G) || a.rows * a.D >= 1LL << 25))
          return launch<T, G, E, VEC, false>();
      return launch<T, G, E, VEC, true>();
    } else {
      return launch<T, G, E, VEC, false>();
    }
  }
  template <typename T, int G, int E, bool VEC, bool AHEAD>
  cudaError_t launch() const {
    using R = Row<T, G, E, VEC>;
    const long long blocks = (a.rows + R::kGroups - 1) / R::kGroups;
    const long long most = AHEAD ? (long long)sm_count() * fwd_blocks<R, AHEAD>() : 1LL << 30;
    return launch_ex(norm_fwd_kernel<T, G, E, VEC, RES, AHEAD>, dim3((unsigned)(blocks < most ? blocks : most)),
                     dim3(R::kThreads), 0, st, 1, (const T *)x, xs, (const T *)res, rs, (const T *)gamma,
                     (const T *)beta, (T *)y, ys, (T *)sum, ss, mean, rstd, a.rows, a.D, a.eps);
  }
};

struct Bwd {
  static constexpr bool kBackward = true, kResidual = false;
  NormArgs a;
  const void *dy, *s, *gamma;
  void *dx;
  long long ys, ss, xs;
  const float *mean, *rstd;
  float *dgamma, *dbeta, *part;
  cudaStream_t st;
  int *partials;  // rows of part that are left to be added

  template <typename T, int G, int E, bool VEC>
  cudaError_t run() const {
    using R = Row<T, G, E, VEC>;
    const long long blocks = (a.rows + R::kGroups - 1) / R::kGroups;
    long long most = (long long)sm_count() * bwd_blocks<R>();
    if (most > kMaxPartials) most = kMaxPartials;
    int grid = (int)(blocks < most ? blocks : most);
    // Two turns of one block's groups at most, of the widest rows one: its sums
    // are the result, and no second launch is needed (us alone and with it: 4 x
    // 1024 bf16 2.3 and 3.4, 8 x 1024 2.9 and 3.6, 12 x 1024 3.4 and 3.5, 2 x
    // 16384 f32 16.0 and 13.6).
    const bool alone = blocks <= (E <= 24 ? 2 : 1) && (!VEC || ((uintptr_t)dgamma | (uintptr_t)dbeta) % 16 == 0);
    if (alone) grid = 1;
    *partials = alone ? 0 : grid;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_shared_on(norm_bwd_kernel<T, G, E, VEC>, bwd_shared<R>(), done);
    if (e != cudaSuccess) return e;
    return launch_ex(norm_bwd_kernel<T, G, E, VEC>, dim3((unsigned)grid), dim3(R::kThreads), bwd_shared<R>(), st, 1,
                     (const T *)dy, ys, (const T *)s, ss, (const T *)gamma, mean, rstd, (T *)dx, xs,
                     alone ? dgamma : part, alone ? dbeta : part + a.D, alone ? 0 : 2 * a.D, a.rows, a.D);
  }
};

// A thread holds 32 bytes of a row (two vectors, in flight together), or 48 of
// widths that would leave lanes idle (forward with residual and backward us,
// with 16 and 24 elements a thread: 65536 x 768 64 and 60, 58 and 50; 20000 x
// 5120 155 and 122, 147 and 125; 9000 x 12000 144 and 134, but 153 and 156; or
// 160 threads: 30000 x 2560 92 and 92, but 55 and 63 without residual, and 85
// and 78, either on 256 100, 66 and 109),
// of the widest rows 64 or 128; narrow rows share a warp (65536 x 200 bf16
// forward: 11.7 us on 16 lanes, 15.7 on a warp). Backward with 8 elements a
// thread: 65536 x 1024 79 us, 68 with 16; with 32, on 384 threads an SM, 63 (81
// on 512, spills), but 8192 x 1024 15.5 against 14.8: longer epilogues.
// Forward without residual, where half as much is in flight: 64 bytes a thread
// (with 32, us: 65536 x 1024 43 and 45, 30000 x 4096 77 and 83, 9000 x 8192 48
// and 61, f32 9000 x 4096 48 and 60), or 48.
template <bool VEC, typename F>
cudaError_t by_width_bf16(const F &f, int D) {
  using T = __nv_bfloat16;
  if constexpr (VEC && !F::kBackward && !F::kResidual) {
    if (D <= 128) return f.template run<T, 8, 16, VEC>();
    if (D <= 256) return f.template run<T, 8, 32, VEC>();
    if (D <= 512) return f.template run<T, 16, 32, VEC>();
    if (D <= 768) return f.template run<T, 32, 24, VEC>();
    if (D <= 1024) return f.template run<T, 32, 32, VEC>();
    if (D <= 1536) return f.template run<T, 64, 24, VEC>();
    if (D <= 2048) return f.template run<T, 64, 32, VEC>();
    if (D <= 2560) return f.template run<T, 128, 24, VEC>();
    if (D <= 4096) return f.template run<T, 128, 32, VEC>();
    if (D <= 6144) return f.template run<T, 256, 24, VEC>();
    if (D <= 8192) return f.template run<T, 256, 32, VEC>();
    if (D <= 12288) return f.template run<T, 512, 24, VEC>();
    return f.template run<T, 512, 32, VEC>();
  } else if constexpr (VEC) {
    if (D <= 128) return f.template run<T, 8, 16, VEC>();
    if (D <= 256) return f.template run<T, 16, 16, VEC>();
    if (D <= 512) return f.template run<T, 32, 16, VEC>();
    if (D <= 768) return f.template run<T, 32, 24, VEC>();
    if constexpr (F::kBackward)
      if (D <= 1024 && f.a.rows >= 16384) return f.template run<T, 32, 32, VEC>();
    if (D <= 1024) return f.template run<T, 64, 16, VEC>();
    if (D <= 1536) return f.template run<T, 64, 24, VEC>();
    if (D <= 2048) return f.template run<T, 128, 16, VEC>();
    if (D <= 2560) {
      if constexpr (F::kBackward) return f.template run<T, 128, 24, VEC>();
      else return f.template run<T, 160, 16, VEC>();
    }
    if (D <= 4096) return f.template run<T, 256, 16, VEC>();
    if (D <= 6144) return f.template run<T, 256, 24, VEC>();
    if (D <= 8192) return f.template run<T, 512, 16, VEC>();
    if constexpr (!F::kBackward)
      if (D <= 12288) return f.template run<T, 512, 24, VEC>();
    return f.template run<T, 512, 32, VEC>();
  } else {
    // single elements: 8 a thread in the forward, which needs no spills (20000 x 2047: 67 us, 84 with 16)
    constexpr int E = F::kBackward ? 16 : 8;
    if (D <= 128) return f.template run<T, 128 / E, E, VEC>();
    if (D <= 256) return f.template run<T, 256 / E, E, VEC>();
    if (D <= 512) return f.template run<T, 512 / E, E, VEC>();
    if (D <= 1024) return f.template run<T, 1024 / E, E, VEC>();
    if (D <= 2048) return f.template run<T, 2048 / E, E, VEC>();
    if (D <= 4096) return f.template run<T, 4096 / E, E, VEC>();
    if (D <= 8192) return f.template run<T, 512, 16, VEC>();
    return f.template run<T, 512, 32, VEC>();
  }
}
// In float32 a thread holds 32 bytes in the forward with a residual and 64
// without. Backward, by vectors, us
// with 8, 12 and 16 elements: 20000 x 2048 75, -, 77; 9000 x 4096 76, -, 73;
// 20000 x 1536 62, 57, -; 12000 x 2560 75, 62, -; 8000 x 5120 82, 80, 82. By
// single elements 16 (20000 x 1023: 44, 52 with 8).
template <bool VEC, typename F>
cudaError_t by_width_f32(const F &f, int D) {
  using T = float;
  constexpr bool kMore = F::kBackward && VEC, kPlain = VEC && !F::kBackward && !F::kResidual;
  constexpr int E = (F::kBackward && !VEC) || kPlain ? 16 : 8;
  if (D <= 128) return f.template run<T, 128 / E, E, VEC>();
  if (D <= 256) return f.template run<T, 256 / E, E, VEC>();
  if (D <= 512) return f.template run<T, 512 / E, E, VEC>();
  if constexpr (kMore)
    if (D <= 768) return f.template run<T, 64, 12, VEC>();
  if (D <= 1024) return f.template run<T, 1024 / E, E, VEC>();
  if constexpr (kMore)
    if (D <= 1536) return f.template run<T, 128, 12, VEC>();
  if (D <= 2048) return f.template run<T, 2048 / E, E, VEC>();
  if constexpr (kMore)
    if (D <= 2560) return f.template run<T, 256, 12, VEC>();
  constexpr int W = F::kBackward || kPlain ? 16 : 8;
  if (D <= 4096) return f.template run<T, 4096 / W, W, VEC>();
  if (D <= 8192) return f.template run<T, 512, 16, VEC>();
  return f.template run<T, 512, 32, VEC>();
}

// Whether all rows start on 16 bytes: the first one, and the stride's rest.
// (Rows that do not go by single elements: 20000 x 1023 f32 forward 50 and
// backward 44 us, 20000 x 1024 by vectors 51 and 41.)
bool starts_whole(const void *p, long long rest) { return (uintptr_t)p % 16 == 0 && rest == 0; }

template <typename F>
cudaError_t dispatch(const F &f, bool vec) {
  if (f.a.dtype == RXL_DTYPE_BF16)
    return vec ? by_width_bf16<true>(f, f.a.D) : by_width_bf16<false>(f, f.a.D);
  return vec ? by_width_f32<true>(f, f.a.D) : by_width_f32<false>(f, f.a.D);
}

}  // namespace

cudaError_t launch_layernorm_fwd(const NormArgs &a, const void *x, long long x_stride, const void *res,
                                 long long res_stride, const void *gamma, const void *beta, void *y,
                                 long long y_stride, void *sum, long long sum_stride, float *mean, float *rstd,
                                 cudaStream_t st, int *launches) {
  const int per = a.dtype == RXL_DTYPE_BF16 ? 8 : 4;
  const auto whole = [&](const void *p, long long stride) { return !p || starts_whole(p, a.rows > 1 ? stride % per : 0); };
  const bool vec = a.D % per == 0 && whole(x, x_stride) && whole(res, res_stride) && whole(y, y_stride) &&
                   whole(sum, sum_stride) && whole(gamma, 0) && whole(beta, 0);
  const auto launch = [&](auto f) { return dispatch(f, vec); };
  const cudaError_t e =
      res ? launch(Fwd<true>{a, x, res, gamma, beta, y, sum, x_stride, res_stride, y_stride, sum_stride, mean, rstd, st})
          : launch(Fwd<false>{a, x, res, gamma, beta, y, sum, x_stride, res_stride, y_stride, sum_stride, mean, rstd, st});
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaGetLastError();
}

size_t layernorm_bwd_workspace(const NormArgs &a) { return ((size_t)kMaxPartials * 2 * a.D * 4 + 15) & ~(size_t)15; }

cudaError_t launch_layernorm_bwd(const NormArgs &a, const void *dy, long long dy_stride, const void *s,
                                 long long s_stride, const void *gamma, const float *mean, const float *rstd,
                                 void *dx, long long dx_stride, float *dgamma, float *dbeta, void *ws,
                                 cudaStream_t st, int *launches) {
  int partials = 0;
  if (a.rows > 0) {
    const int per = a.dtype == RXL_DTYPE_BF16 ? 8 : 4;
    const auto whole = [&](const void *p, long long stride) { return starts_whole(p, a.rows > 1 ? stride % per : 0); };
    const bool vec = a.D % per == 0 && whole(dy, dy_stride) && whole(s, s_stride) && whole(dx, dx_stride) && whole(gamma, 0);
    const Bwd f = {a, dy, s, gamma, dx, dy_stride, s_stride, dx_stride, mean, rstd, dgamma, dbeta, (float *)ws, st, &partials};
    const cudaError_t e = dispatch(f, vec);
    if (e != cudaSuccess) return e;
    ++*launches;
    if (partials == 0) return cudaGetLastError();
  }
  const int columns = a.D <= 2048 && partials > 152 ? 8 : 32;
  const cudaError_t e = launch_ex(columns == 8 ? norm_bwd_join_kernel<8> : norm_bwd_join_kernel<32>,
                                  dim3((2 * a.D + columns - 1) / columns), dim3(kJoinThreads), 0, st, 1,
                                  (const float *)ws, dgamma, dbeta, partials, a.D);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaGetLastError();
}

}  // namespace rxl
