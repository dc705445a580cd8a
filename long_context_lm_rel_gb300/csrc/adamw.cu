// One AdamW step over a list of tensors, states in 32 or 8 bits
// (include/rxl.h: rxl_adamw_step).
//
// Memory-bound: every operand is read once and written once (28 bytes an
// element for bf16 weights with masters and 32-bit states, 16.13 for f32
// weights, f32 gradients and 8-bit states). The list travels in the kernel's
// parameters (up to kPerLaunch tensors a launch, so a 16-layer stack is one
// launch); a tensor is cut into chunks of 1024 elements, one a block, and a
// block finds its tensor in a small table of the chunks' high bits (a
// bisection of the running count cost 5% in 8 bits). A thread takes 8
// consecutive elements, all of whose operands it loads before it uses any, so
// that 1024 threads an SM keep ~100 KB in flight.
//
// 32 bits (201 M bf16 weights with masters, 224 tensors): 794 us, 7.10 TB/s, a
// little above the copy rate the card was measured at.
//
// In 8 bits the 128 elements that share a scale belong to 16 lanes, whose
// largest magnitudes meet in four shuffles. The exact square root, the exact
// quotient and the rounding by chance make about a hundred instructions an
// element, which bounds it whatever the bytes are: 72 us for 25 M f32 weights
// (5.6 TB/s of 16.13 bytes an element), 78 for bf16 ones with masters (5.2) and
// 78 for bf16 alone (3.3 of 10.13); 201 M: 550, 593 and 591 us. At 48 registers
// each of these kernels stores 48 to 56 bytes a thread to local memory.
// Sixteen elements a thread: 102 us (registers); 8, 9 or 11 blocks an SM
// instead of 10: 72 and 634, 70 and 605, 75 and 609; blocks of 256 threads: 74
// and 612; blocks that take chunks in turn: 2 more.
#include <cuda_fp8.h>
#include <math.h>

#include "sm103.cuh"
#include "stream_common.cuh"
#include "train.cuh"

namespace rxl {
namespace {

using namespace stream;
using sm103::griddep_launch_dependents;
using sm103::griddep_wait;

constexpr int kBlock = 128;  // elements that share a scale
constexpr int kThreads = 128;
constexpr int kPer = 8;      // consecutive elements of a thread
constexpr int kChunk = kThreads * kPer;
constexpr int kPerLaunch = 384;

struct Entry {
  void *param;
  float *master;
  const void *grad;
  void *m, *v;
  float *m_scale, *v_scale;
  long long n;
  float weight_decay;
  unsigned index;  // place in the caller's list
};

constexpr int kMap = 512;

struct Step {
  Entry t[kPerLaunch];
  long long first[kPerLaunch + 1];  // chunks before tensor i
  unsigned short map[kMap];         // the tensor of chunk i << shift
  int n, shift;
  float beta1, beta2, one_beta1, one_beta2, eps;
  rxl_adamw_scalars s;
  const rxl_adamw_scalars *dev;
};
static_assert(sizeof(Step) <= 32764, "the list is a kernel parameter");

__device__ __forceinline__ unsigned dither(unsigned i, unsigned key) {
  unsigned h = i * 0x9E3779B1u + key;
  h = (h ^ (h >> 16)) * 0x9E3779B1u;
  h = (h ^ (h >> 15)) * 0x85157AF5u;
  return h ^ (h >> 16);
}

// 0 <= a <= 448 (1 + 2^-23) to e4m3 values, up with the probability of what is cut off:
// random bits (c: 16, added at the place of the first ones that are cut)
// below the kept mantissa, or, below the normal range, to the multiple of the
// step 2^-9 there. That second case is rare (2^-15 of the block's largest and
// less, or NaN, which stays) and has a branch of its own for all of them.
// POSITIVE: what is above 0 stays so. A block's largest is 448 but for two
// roundings, and becomes 448: above it the last place and 16 bits carry no
// further; a place or two below it they carry to 448, but for 16 random bits
// that are all 0 (2^-16: 416, the code below).
template <bool POSITIVE>
__device__ __forceinline__ void chance_e4m3(const float (&a)[kPer], const unsigned (&c)[kPer], float (&q)[kPer]) {
  static_assert(kPer == 8);
  const float least = min_nan(min_nan(a[0], a[1], a[2]), min_nan(a[3], a[4], a[5]), min_nan(a[6], a[7], a[7]));
#pragma unroll
  for (int k = 0; k < kPer; ++k) q[k] = __uint_as_float((__float_as_uint(a[k]) + (c[k] << 4)) & 0xFFF00000u);
  if (!(least >= 0x1p-6f)) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (!(a[k] >= 0x1p-6f)) q[k] = floorf(__fadd_rn(a[k] * 512.f, (float)c[k] * 0x1p-16f)) * 0x1p-9f;
      if (POSITIVE && a[k] > 0.f) q[k] = max_nan(q[k], 0x1p-9f);
    }
  }
}

// kPer consecutive elements: whole vectors, or element by element at a
// tensor's end (cnt of them; the others are 0).
template <typename T>
__device__ __forceinline__ void read(const T *p, int cnt, float (&v)[kPer]) {
  if (cnt == kPer) {
#pragma unroll
    for (int i = 0; i < kPer / kVec<T>; ++i) {
      float f[kVec<T>];
      unpack(*((const uint4 *)p + i), f);
#pragma unroll
      for (int k = 0; k < kVec<T>; ++k) v[i * kVec<T> + k] = f[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = k < cnt ? to_f32(p[k]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void write(T *p, int cnt, const float (&v)[kPer]) {
  if (cnt == kPer) {
#pragma unroll
    for (int i = 0; i < kPer / kVec<T>; ++i) {
      float f[kVec<T>];
#pragma unroll
      for (int k = 0; k < kVec<T>; ++k) f[k] = v[i * kVec<T> + k];
      *((uint4 *)p + i) = pack(f);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (k < cnt) p[k] = from_f32<T>(v[k]);
  }
}

// e4m3 codes, four to a word.
struct Codes {
  uint32_t w[kPer / 4];
  __device__ __forceinline__ void read(const unsigned char *p, int cnt) {
    if (cnt == kPer) {
      const uint2 u = *(const uint2 *)p;
      w[0] = u.x;
      w[1] = u.y;
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (k % 4 == 0) w[k / 4] = 0;
        if (k < cnt) w[k / 4] |= (uint32_t)p[k] << (8 * (k % 4));
      }
    }
  }
  __device__ __forceinline__ void write(unsigned char *p, int cnt) const {
    if (cnt == kPer) {
      *(uint2 *)p = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (k < cnt) p[k] = (unsigned char)(w[k / 4] >> (8 * (k % 4)));
    }
  }
  __device__ __forceinline__ void values(float scale, float (&v)[kPer]) const {
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
      const __half2_raw h =
          __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k / 4] >> (8 * (k % 4))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[k] = __fmul_rn(f.x, scale);
      v[k + 1] = __fmul_rn(f.y, scale);
    }
  }
  __device__ __forceinline__ void encode(const float (&q)[kPer]) {
#pragma unroll
    for (int k = 0; k < kPer; k += 4) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[k], q[k + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[k + 2], q[k + 3]), __NV_SATFINITE, __NV_E4M3);
      w[k / 4] = lo | hi << 16;
    }
  }
};

// Every operation is rounded on its own (no contraction: packed pairs are
// not used here, which the assembler contracts), in the order include/rxl.h
// gives.
template <typename P, typename G, bool MASTER, bool EIGHT>
__global__ void __launch_bounds__(kThreads, EIGHT ? 10 : 8) adamw_kernel(const __grid_constant__ Step step) {
  griddep_wait();
  griddep_launch_dependents();
  const rxl_adamw_scalars s = step.dev ? *step.dev : step.s;
  const long long b = blockIdx.x;
  int at = step.map[b >> step.shift];
  while (b >= step.first[at + 1]) ++at;
  const Entry &t = step.t[at];
  const long long i = (b - step.first[at]) * kChunk + (int)threadIdx.x * kPer;
  const long long left = t.n - i;
  const int cnt = left >= kPer ? kPer : left > 0 ? (int)left : 0;
  float g[kPer], w[kPer], m[kPer], v[kPer], r[kPer];
  Codes cm, cv;
  float sm = 0.f, sv = 0.f;
  read((const G *)t.grad + i, cnt, g);
  if (MASTER) read(t.master + i, cnt, w);
  else read((const P *)t.param + i, cnt, w);
  if (EIGHT) {
    cm.read((const unsigned char *)t.m + i, cnt);
    cv.read((const unsigned char *)t.v + i, cnt);
    if (cnt) {
      sm = t.m_scale[i / kBlock];
      sv = t.v_scale[i / kBlock];
    }
    cm.values(sm, m);
    cv.values(sv, v);
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = __fmul_rn(v[k], v[k]);
  } else {
    read((const float *)t.m + i, cnt, m);
    read((const float *)t.v + i, cnt, v);
  }
  const float keep = __fsub_rn(1.f, __fmul_rn(s.lr, t.weight_decay));
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const float gk = __fmul_rn(g[k], s.grad_scale);
    m[k] = __fadd_rn(__fmul_rn(m[k], step.beta1), __fmul_rn(gk, step.one_beta1));
    v[k] = __fadd_rn(__fmul_rn(v[k], step.beta2), __fmul_rn(__fmul_rn(gk, step.one_beta2), gk));
    r[k] = __fsqrt_rn(v[k]);
    const float u =
        __fdiv_rn(__fmul_rn(m[k], s.m_correction), __fadd_rn(__fmul_rn(r[k], s.v_correction), step.eps));
    w[k] = __fsub_rn(__fmul_rn(w[k], keep), __fmul_rn(u, s.lr));
  }
  if (MASTER) write(t.master + i, cnt, w);
  write((P *)t.param + i, cnt, w);
  if (!EIGHT) {
    write((float *)t.m + i, cnt, m);
    write((float *)t.v + i, cnt, v);
  } else {
    // Elements beyond the tensor are 0 here. NaN is left out: it spoils its
    // own code only.
    float tm = 0.f, tr = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
      tm = max3(tm, fabsf(m[k]), fabsf(m[k + 1]));
      tr = max3(tr, r[k], r[k + 1]);
    }
#pragma unroll
    for (int o = kBlock / kPer / 2; o > 0; o >>= 1) {
      tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
      tr = fmaxf(tr, __shfl_xor_sync(0xffffffffu, tr, o));
    }
    const bool fm = tm >= 0x1p-100f, fr = tr >= 0x1p-100f;
    const float im = fm ? __fdiv_rn(448.f, tm) : 0.f, ir = fr ? __fdiv_rn(448.f, tr) : 0.f;
    const unsigned key = s.seed * 0x85157AF5u + t.index * 0xC2B2AE3Du;
    float q[kPer], a[kPer];
    unsigned h[kPer], c[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      h[k] = dither((unsigned)i + k, key);
      c[k] = h[k] & 0xFFFFu;
      a[k] = __fmul_rn(fabsf(m[k]), im);
    }
    chance_e4m3<false>(a, c, q);
#pragma unroll
    for (int k = 0; k < kPer; ++k) q[k] = copysignf(q[k], m[k]);
    cm.encode(q);
    cm.write((unsigned char *)t.m + i, cnt);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      c[k] = h[k] >> 16;
      a[k] = __fmul_rn(r[k], ir);
    }
    chance_e4m3<true>(a, c, q);
    cv.encode(q);
    cv.write((unsigned char *)t.v + i, cnt);
    if (cnt && i % kBlock == 0) {
      t.m_scale[i / kBlock] = fm ? __fmul_rn(tm, (float)(1.0 / 448)) : 0.f;
      t.v_scale[i / kBlock] = fr ? __fmul_rn(tr, (float)(1.0 / 448)) : 0.f;
    }
  }
}

using Kernel = void (*)(Step);

template <typename P, typename G, bool MASTER>
Kernel pick_bits(bool eight) {
  return eight ? adamw_kernel<P, G, MASTER, true> : adamw_kernel<P, G, MASTER, false>;
}
template <typename P, bool MASTER>
Kernel pick_grad(rxl_dtype g, bool eight) {
  return g == RXL_DTYPE_BF16 ? pick_bits<P, __nv_bfloat16, MASTER>(eight) : pick_bits<P, float, MASTER>(eight);
}

}  // namespace

cudaError_t launch_adamw(const rxl_adamw_desc &d, const rxl_adamw_tensor *tensors, int n,
                         const rxl_adamw_scalars &scalars, const rxl_adamw_scalars *scalars_dev, cudaStream_t st,
                         int *launches) {
  const bool eight = d.state_bits == 8;
  Step step;
  step.beta1 = d.beta1;
  step.beta2 = d.beta2;
  step.one_beta1 = (float)(1.0 - (double)d.beta1);
  step.one_beta2 = (float)(1.0 - (double)d.beta2);
  step.eps = d.eps;
  step.s = scalars;
  step.dev = scalars_dev;
  for (int i = 0; i < n;) {
    step.n = 0;
    step.first[0] = 0;
    bool master = false;
    for (; i < n && step.n < kPerLaunch; ++i) {
      const rxl_adamw_tensor &t = tensors[i];
      if (t.n == 0) continue;
      step.t[step.n] = {t.param, t.master, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.n, t.weight_decay, (unsigned)i};
      master = t.master != nullptr;
      step.first[step.n + 1] = step.first[step.n] + (t.n + kChunk - 1) / kChunk;
      ++step.n;
    }
    if (step.n == 0) break;
    // A block looks its tensor up by its chunk's high bits and goes on from
    // there.
    const long long chunks = step.first[step.n];
    for (step.shift = 0; (chunks - 1) >> step.shift >= kMap; ++step.shift) {
    }
    for (int k = 0, at = 0; k <= (int)((chunks - 1) >> step.shift); ++k) {
      while ((long long)k << step.shift >= step.first[at + 1]) ++at;
      step.map[k] = (unsigned short)at;
    }
    const Kernel k = d.param_dtype == RXL_DTYPE_F32 ? pick_grad<float, false>(d.grad_dtype, eight)
                     : master                       ? pick_grad<__nv_bfloat16, true>(d.grad_dtype, eight)
                                                    : pick_grad<__nv_bfloat16, false>(d.grad_dtype, eight);
    // a block for every chunk: the entry point admits 2^40 elements, 2^30 chunks and a few
    const cudaError_t e = launch_ex(k, dim3((unsigned)chunks), dim3(kThreads), 0, st, 1, step);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return *launches ? cudaGetLastError() : cudaSuccess;
}

}  // namespace rxl
