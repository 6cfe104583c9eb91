// Gradient norms and clipping for gfx950: the global norm over many tensors, the
// scaling that limits it, and both inside the Allreduce of P rank buffers.
//
//   N     = sqrt(sum over every element of g^2), or the largest |g|
//   scale = 1 where N + eps <= max_norm, else max_norm / (N + eps)
//   y     = scale g, rounded once to y's type
//
// Every pass streams memory; the arithmetic per element is a widening, a
// multiply-add in 64 bits and one multiplication. Tensors are cut into work items
// of `per` elements; an item's partial norm is one 64-bit value at its own place,
// and the partials are combined in their order, so a list of the same sizes gives
// the same bits whatever runs beside it.
//
// Squares are summed in 64 bits: fp32 squares overflow from 1.8e19 on, and a sum
// over 10^9 elements has no bits left in 24. Largest magnitudes compare the
// magnitudes' bit patterns as integers, which orders NaN above infinity, so a NaN
// anywhere is the result.
#include "grad.h"

#include <hip/hip_ext.h>

#include <algorithm>
#include <cstring>
#include <map>
#include <mutex>
#include <vector>

#include "kernels.h"
#include "launch.h"

namespace ar {

// ----------------------------------------------------------------------------
// arithmetic
// ----------------------------------------------------------------------------
// Vectors of 16 bytes at any element's address: global accesses of this target
// need no alignment, and a tensor's vectors are counted from its first element, so
// how it is cut (and the order of its sums) does not depend on where it lies.
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));

// fp32 -> bf16 bits, to nearest even; NaN stays NaN (a carry out of a NaN's
// payload would make it an infinity or a zero).
__device__ __forceinline__ uint32_t bf16_of(float f) {
  const uint32_t u = as_u(f);
  const uint32_t r = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
  return (u & 0x7fffffffu) > 0x7f800000u ? (u >> 16) | 0x40u : r;
}

template <int DT, int V> __device__ __forceinline__ void ld_unit(const void* base, int64_t e, float (&x)[V]) {
  if constexpr (DT == D_BF16) {
    static_assert(V == 8, "8 bf16 to a vector");
    const u32x4_e2 r = *reinterpret_cast<const u32x4_e2*>(static_cast<const uint16_t*>(base) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = as_f(r[i] << 16);
      x[2 * i + 1] = as_f(r[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const u32x4_e4 r = *(reinterpret_cast<const u32x4_e4*>(static_cast<const float*>(base) + e) + q);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * q + i] = as_f(r[i]);
    }
  }
}

template <int DT, int V> __device__ __forceinline__ void st_unit(void* base, int64_t e, const float (&x)[V]) {
  if constexpr (DT == D_BF16) {
    static_assert(V == 8, "8 bf16 to a vector");
    u32x4_e2 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = bf16_of(x[2 * i]) | (bf16_of(x[2 * i + 1]) << 16);
    *reinterpret_cast<u32x4_e2*>(static_cast<uint16_t*>(base) + e) = r;
  } else {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      u32x4_e4 r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = as_u(x[4 * q + i]);
      *(reinterpret_cast<u32x4_e4*>(static_cast<float*>(base) + e) + q) = r;
    }
  }
}

template <int DT> __device__ __forceinline__ float ld_one(const void* base, int64_t e) {
  if constexpr (DT == D_BF16) return as_f(uint32_t(static_cast<const uint16_t*>(base)[e]) << 16);
  else return static_cast<const float*>(base)[e];
}

template <int DT> __device__ __forceinline__ void st_one(void* base, int64_t e, float x) {
  if constexpr (DT == D_BF16) static_cast<uint16_t*>(base)[e] = uint16_t(bf16_of(x));
  else static_cast<float*>(base)[e] = x;
}

// A partial norm: the sum of squares, or the largest magnitude, as a double.
template <int KIND> struct Part {
  double v = 0;
  __device__ __forceinline__ void add(float x) {
    if constexpr (KIND == N_L2) {
      const double d = double(x);
      v = __builtin_fma(d, d, v);
    } else {
      join(double(as_f(as_u(x) & 0x7fffffffu)));
    }
  }
  __device__ __forceinline__ void join(double o) {
    if constexpr (KIND == N_L2) {
      v += o;
    } else {
      const uint64_t a = uint64_t(__double_as_longlong(v)), b = uint64_t(__double_as_longlong(o));
      if (b > a) v = o;  // magnitudes: sign bits are clear
    }
  }
  __device__ __forceinline__ double norm() const {
    if constexpr (KIND == N_L2) return sqrt(v);
    else return v;
  }
};

// The workgroup's partial, valid in thread 0: within a wave by shuffles, then over the waves in order.
template <int KIND, int THREADS> __device__ __forceinline__ void join_group(Part<KIND>& p) {
  __shared__ double wave[THREADS / 64];
#pragma unroll
  for (int d = 32; d; d >>= 1) p.join(__shfl_down(p.v, d));
  __syncthreads();  // the array's last readers
  if (threadIdx.x % 64 == 0) wave[threadIdx.x / 64] = p.v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < THREADS / 64; ++w) p.join(wave[w]);
}

// The scale as a product a b of two fp32 values: one where it has fp32's full precision, and below
// 2^-64 (a limit far under an exploding norm) two halves of its exponent, so that x a b is right for
// every x and rounds once more only where the result has no 24 bits.
struct Factor {
  float a, b;
  __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};

__device__ __forceinline__ Factor factor_of(double norm, float max_norm, float eps) {
  const double reach = norm + double(eps);
  const double s = reach <= double(max_norm) ? 1.0 : double(max_norm) / reach;  // a NaN stays one
  if (s > 0 && s < 0x1p-64) {
    int e;
    const double m = frexp(s, &e);
    const int ea = max(e / 2, -125);
    return {float(ldexp(m, ea)), float(ldexp(1.0, e - ea))};
  }
  return {float(s), 1.0f};
}

// ----------------------------------------------------------------------------
// tensor lists
// ----------------------------------------------------------------------------
// A launch's tensors, passed by value: the caller's list may change after the call, a captured call
// carries its own, and nothing is copied to the device. 4 KB of arguments hold 128 tensors; longer
// lists take several launches.
constexpr int kTabTensors = 128;
struct GradTab {
  const void* src[kTabTensors];
  void* dst[kTabTensors];
  int64_t n4[kTabTensors];         // elements << 2 | out is bf16 << 1 | data is bf16
  int32_t first[kTabTensors + 1];  // first work item of every tensor, from 0
  int32_t count;
  int32_t at;   // place of item 0 among the call's partials
  int64_t per;  // elements per work item
};
static_assert(sizeof(GradTab) <= 4000, "kernel arguments");

// The tensor an item belongs to: the last whose first item is not past it (tensors without elements
// share the next one's first item).
template <typename TAB> __device__ __forceinline__ int find_first(const TAB& tab, int count, int item) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (tab.first[mid] <= item) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int KIND, int DT> __device__ __forceinline__ void norm_item(const void* src, int64_t e0, int64_t cnt, Part<KIND>& p) {
  constexpr int V = DT == D_BF16 ? 8 : 4;
  const int64_t nv = cnt / V;
  for (int64_t v = threadIdx.x; v < nv; v += kThreads) {
    float x[V];
    ld_unit<DT, V>(src, e0 + v * V, x);
#pragma unroll
    for (int i = 0; i < V; ++i) p.add(x[i]);
  }
  const int64_t t = nv * V + threadIdx.x;
  if (t < cnt) p.add(ld_one<DT>(src, e0 + t));
}

template <int KIND> __global__ __launch_bounds__(kThreads) void k_grad_norm(GradTab tab, double* partial) {
  for (int it = blockIdx.x; it < tab.first[tab.count]; it += gridDim.x) {
    const int i = find_first(tab, tab.count, it);
    const int64_t n = tab.n4[i] >> 2, e0 = (it - tab.first[i]) * tab.per, cnt = min(tab.per, n - e0);
    Part<KIND> p;
    if (tab.n4[i] & 1) norm_item<KIND, D_BF16>(tab.src[i], e0, cnt, p);
    else norm_item<KIND, D_FP32>(tab.src[i], e0, cnt, p);
    join_group<KIND, kThreads>(p);
    if (threadIdx.x == 0) partial[tab.at + it] = p.v;
  }
}

constexpr int kFinalThreads = 1024;
template <int KIND> __global__ __launch_bounds__(kFinalThreads) void k_norm_final(const double* partial, int items, double* norm, float* total) {
  Part<KIND> p;
  for (int i = threadIdx.x; i < items; i += kFinalThreads) p.join(partial[i]);
  join_group<KIND, kFinalThreads>(p);
  if (threadIdx.x == 0) {
    *norm = p.norm();
    if (total) *total = float(p.norm());
  }
}

constexpr int kEachTensors = 900;
struct EachTab {
  int32_t first[kEachTensors + 1];  // first partial of every tensor
};

template <int KIND> __global__ __launch_bounds__(64) void k_norm_each(EachTab tab, const double* partial, float* each) {
  const int i = blockIdx.x;
  Part<KIND> p;
  for (int k = tab.first[i] + threadIdx.x; k < tab.first[i + 1]; k += 64) p.join(partial[k]);
  join_group<KIND, 64>(p);
  if (threadIdx.x == 0) each[i] = float(p.norm());
}

template <int DS, int DD> __device__ __forceinline__ void scale_item(const void* src, void* dst, int64_t e0, int64_t cnt, Factor f) {
  constexpr int V = DS == D_BF16 || DD == D_BF16 ? 8 : 4;
  const int64_t nv = cnt / V;
  for (int64_t v = threadIdx.x; v < nv; v += kThreads) {
    float x[V];
    ld_unit<DS, V>(src, e0 + v * V, x);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = f(x[i]);
    st_unit<DD, V>(dst, e0 + v * V, x);
  }
  const int64_t t = nv * V + threadIdx.x;
  if (t < cnt) st_one<DD>(dst, e0 + t, f(ld_one<DS>(src, e0 + t)));
}

__global__ __launch_bounds__(kThreads) void k_grad_scale(GradTab tab, const double* norm, const float* known, float max_norm, float eps) {
  const Factor f = factor_of(known ? double(*known) : *norm, max_norm, eps);
  for (int it = blockIdx.x; it < tab.first[tab.count]; it += gridDim.x) {
    const int i = find_first(tab, tab.count, it);
    const int64_t n = tab.n4[i] >> 2, e0 = (it - tab.first[i]) * tab.per, cnt = min(tab.per, n - e0);
    const void* s = tab.src[i];
    void* d = tab.dst[i];
    switch (int(tab.n4[i] & 3)) {
      case 0: scale_item<D_FP32, D_FP32>(s, d, e0, cnt, f); break;
      case 1: scale_item<D_BF16, D_FP32>(s, d, e0, cnt, f); break;
      case 2: scale_item<D_FP32, D_BF16>(s, d, e0, cnt, f); break;
      default: scale_item<D_BF16, D_BF16>(s, d, e0, cnt, f); break;
    }
  }
}

// ----------------------------------------------------------------------------
// the Allreduce that clips
// ----------------------------------------------------------------------------
// Two passes over the element range, with the norm between them. The first reads all P buffers,
// combines them in rank order (the direct schedule's order and roundings), takes the norm of the
// sums and leaves them, in full fp32, where the second finds them; the second scales them, rounds
// once and writes them to every rank: (2 P + 2) elements moved for the Allreduce's own 2 P.
//
// The sums lie in the result's own place: fp32 sums in rank 0's buffer (the Allreduce), or in the
// owner's part (the reduce-scatter); a bf16 sum's upper half there and its lower half at the same
// place of rank 1's buffer, or of the workspace (the reduce-scatter leaves other elements alone).
// With one rank the sum is its only operand and has no lower half.
constexpr int kTabPtrs = 400, kTabBuckets = 16;
struct BucketTab {
  void* p[kTabPtrs];               // P pointers of every bucket
  uint16_t* low[kTabBuckets];      // lower halves of bf16 sums, by element; null: none
  int64_t part[kTabBuckets];       // elements per part (the whole bucket for the Allreduce)
  int64_t n[kTabBuckets];
  int32_t first[kTabBuckets + 1];  // first work item
  int32_t ipp[kTabBuckets];        // work items per part
  int32_t count, P, at;
  int32_t owners;                  // 1: part q belongs to rank q alone
  int64_t per;
  float div;                       // > 0: the sum is divided by it
};
static_assert(sizeof(BucketTab) <= 4000, "kernel arguments");

struct BucketItem {
  int b, owner;
  int64_t e0, cnt;
};

__device__ __forceinline__ BucketItem bucket_item(const BucketTab& tab, int it) {
  BucketItem r;
  r.b = find_first(tab, tab.count, it);
  const int k = it - tab.first[r.b], q = k / tab.ipp[r.b];
  r.owner = tab.owners ? q : 0;
  const int64_t lo = q * tab.part[r.b], hi = min(lo + tab.part[r.b], tab.n[r.b]);
  r.e0 = lo + (k - q * tab.ipp[r.b]) * tab.per;
  r.cnt = max(int64_t(0), min(tab.per, hi - r.e0));  // the last parts may be short or empty
  return r;
}

// The ranks' vectors are read once, in batches of B ranks whose loads are all in flight before the first
// is added; a thread's M vectors go together. One load at a time took 135 us for the sums of 7 x 2^24
// fp32 and 134 us for those of 192 x 2^20 bf16; loading the next batch before adding this one gained
// nothing (178 and 132 us for the whole call, against 175 and 135).
template <int DT> struct Raw;
template <> struct Raw<D_FP32> { using T = u32x4_e4; };
template <> struct Raw<D_BF16> { using T = u32x4_e2; };

template <int DT, int V, int M, int B>
__device__ __forceinline__ void ld_ranks(void* const* ptr, int P, int base, int64_t e, const bool (&ok)[M], u32x4 (&r)[B][M]) {
#pragma unroll
  for (int k = 0; k < B; ++k) {
    const typename TT<DT>::S* p = static_cast<const typename TT<DT>::S*>(ptr[base + k < P ? base + k : base]) + e;
#pragma unroll
    for (int j = 0; j < M; ++j)
      if (ok[j]) r[k][j] = __builtin_nontemporal_load(reinterpret_cast<const typename Raw<DT>::T*>(p + j * kThreads * V));
  }
}

template <int DT, int V, int M, int B>
__device__ __forceinline__ void add_ranks(int P, int base, const u32x4 (&r)[B][M], float (&acc)[M][V]) {
#pragma unroll
  for (int k = 0; k < B; ++k) {
    if (base + k >= P) continue;
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float x = DT == D_FP32 ? as_f(r[k][j][i % 4])
                                     : as_f(i % 2 ? r[k][j][i / 2] & 0xffff0000u : r[k][j][i / 2] << 16);
        acc[j][i] = base + k ? acc[j][i] + x : x;
      }
  }
}

template <int DT, int V, int M, int B>
__device__ __forceinline__ void sum_ranks(void* const* ptr, int P, float div, int64_t e, const bool (&ok)[M], float (&acc)[M][V]) {
  for (int base = 0; base < P; base += B) {
    u32x4 r[B][M];
    ld_ranks<DT, V, M, B>(ptr, P, base, e, ok, r);
    add_ranks<DT, V, M, B>(P, base, r, acc);
  }
  if (div > 0) {
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[j][i] = acc[j][i] / div;
  }
}

template <int DT> __device__ __forceinline__ float sum_one(void* const* ptr, int P, float div, int64_t e) {
  float acc = ld_one<DT>(ptr[0], e);
  for (int q = 1; q < P; ++q) acc = acc + ld_one<DT>(ptr[q], e);
  return div > 0 ? acc / div : acc;
}

// Whole sums to and from their place.
template <int DT, int V> __device__ __forceinline__ void put_sum(void* own, uint16_t* low, int64_t e, const float (&s)[V]) {
  if constexpr (DT == D_FP32) {
    if constexpr (V == 1) static_cast<float*>(own)[e] = s[0];
    else st_unit<D_FP32, V>(own, e, s);
  } else if constexpr (V == 1) {
    static_cast<uint16_t*>(own)[e] = uint16_t(as_u(s[0]) >> 16);
    if (low) low[e] = uint16_t(as_u(s[0]));
  } else {
    u32x4_e2 h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = as_u(s[2 * i]), b = as_u(s[2 * i + 1]);
      h[i] = (a >> 16) | (b & 0xffff0000u);
      l[i] = (a & 0xffffu) | (b << 16);
    }
    *reinterpret_cast<u32x4_e2*>(static_cast<uint16_t*>(own) + e) = h;
    if (low) *reinterpret_cast<u32x4_e2*>(low + e) = l;
  }
}

template <int DT, int V> __device__ __forceinline__ void get_sum(const void* own, const uint16_t* low, int64_t e, float (&s)[V]) {
  if constexpr (DT == D_FP32) {
    if constexpr (V == 1) s[0] = static_cast<const float*>(own)[e];
    else ld_unit<D_FP32, V>(own, e, s);
  } else if constexpr (V == 1) {
    s[0] = as_f((uint32_t(static_cast<const uint16_t*>(own)[e]) << 16) | (low ? low[e] : 0u));
  } else {
    const u32x4_e2 h = *reinterpret_cast<const u32x4_e2*>(static_cast<const uint16_t*>(own) + e);
    u32x4_e2 l = {0, 0, 0, 0};
    if (low) l = *reinterpret_cast<const u32x4_e2*>(low + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[2 * i] = as_f((h[i] << 16) | (l[i] & 0xffffu));
      s[2 * i + 1] = as_f((h[i] & 0xffff0000u) | (l[i] >> 16));
    }
  }
}

template <int DT, int KIND, int B>
__global__ __launch_bounds__(kThreads) void k_bucket_reduce(BucketTab tab, double* partial) {
  constexpr int V = DT == D_BF16 ? 8 : 4, M = 8 / V;
  for (int it = blockIdx.x; it < tab.first[tab.count]; it += gridDim.x) {
    const BucketItem w = bucket_item(tab, it);
    void* const* ptr = tab.p + w.b * tab.P;
    Part<KIND> p;
    const int64_t nv = w.cnt / V;
    for (int64_t v = threadIdx.x; v < nv; v += kThreads * M) {
      bool ok[M];
#pragma unroll
      for (int j = 0; j < M; ++j) ok[j] = v + j * kThreads < nv;
      float s[M][V];
      sum_ranks<DT, V, M, B>(ptr, tab.P, tab.div, w.e0 + v * V, ok, s);
#pragma unroll
      for (int j = 0; j < M; ++j)
        if (ok[j]) {
#pragma unroll
          for (int i = 0; i < V; ++i) p.add(s[j][i]);
          put_sum<DT, V>(ptr[w.owner], tab.low[w.b], w.e0 + (v + j * kThreads) * V, s[j]);
        }
    }
    const int64_t t = nv * V + threadIdx.x;
    if (t < w.cnt) {
      const float s[1] = {sum_one<DT>(ptr, tab.P, tab.div, w.e0 + t)};
      p.add(s[0]);
      put_sum<DT, 1>(ptr[w.owner], tab.low[w.b], w.e0 + t, s);
    }
    join_group<KIND, kThreads>(p);
    if (threadIdx.x == 0) partial[tab.at + it] = p.v;
  }
}

// Items go in the first pass's order, workgroup by workgroup: the sums are then read on the XCD that
// wrote them, and out of its L2 or the cache in front of HBM (7 x 2^24 fp32: 173 us for the call, 184 us in
// the opposite order; 8 x 2^20: 25 and 31 us).
template <int DT> __global__ __launch_bounds__(kThreads) void k_bucket_spread(BucketTab tab, const double* norm, float max_norm, float eps) {
  constexpr int V = DT == D_BF16 ? 8 : 4, M = 8 / V;
  const Factor f = factor_of(*norm, max_norm, eps);
  for (int it = blockIdx.x; it < tab.first[tab.count]; it += gridDim.x) {
    const BucketItem w = bucket_item(tab, it);
    void* const* ptr = tab.p + w.b * tab.P;
    const int q0 = tab.owners ? w.owner : 0, q1 = tab.owners ? w.owner + 1 : tab.P;
    const int64_t nv = w.cnt / V;
    for (int64_t v = threadIdx.x; v < nv; v += kThreads * M) {
      bool ok[M];
      float s[M][V];
#pragma unroll
      for (int j = 0; j < M; ++j) {
        ok[j] = v + j * kThreads < nv;
        if (ok[j]) get_sum<DT, V>(ptr[w.owner], tab.low[w.b], w.e0 + (v + j * kThreads) * V, s[j]);
      }
#pragma unroll
      for (int j = 0; j < M; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s[j][i] = f(s[j][i]);
      for (int q = q0; q < q1; ++q)
#pragma unroll
        for (int j = 0; j < M; ++j)
          if (ok[j]) st_unit<DT, V>(ptr[q], w.e0 + (v + j * kThreads) * V, s[j]);
    }
    const int64_t t = nv * V + threadIdx.x;
    if (t < w.cnt) {
      float s[1];
      get_sum<DT, 1>(ptr[w.owner], tab.low[w.b], w.e0 + t, s);
      s[0] = f(s[0]);
      for (int q = q0; q < q1; ++q) st_one<DT>(ptr[q], w.e0 + t, s[0]);
    }
  }
}

// ----------------------------------------------------------------------------
// host
// ----------------------------------------------------------------------------
namespace {

RunResult hip_fail(hipError_t e, const char* what) {
  RunResult r;
  r.status = 4;  // AR_HIP_ERROR
  r.hip_error = int(e);
  r.message = std::string(what) + ": " + hipGetErrorString(e);
  return r;
}

// Work items: at most about kMaxItems, of a multiple of kItemUnit elements.
constexpr int64_t kItemUnit = 2048, kMaxItems = 16384;
int64_t item_size(int64_t total) {
  const int64_t want = (total + kMaxItems - 1) / kMaxItems;
  return std::max(kItemUnit, (want + kItemUnit - 1) / kItemUnit * kItemUnit);
}
int64_t pieces(int64_t n, int64_t per) { return (n + per - 1) / per; }

constexpr size_t kHead = 256;  // the norm, in front of the partials
size_t round_up(size_t b) { return (b + 255) / 256 * 256; }

// Workspaces of calls that bring none. The launches of such a call stay together on its stream: a
// second call on the same stream waits for g_mu, not between this call's passes.
struct Kept {
  void* p = nullptr;
  size_t bytes = 0;
  int device = 0;
};
std::mutex g_mu;
std::map<std::pair<int, uintptr_t>, Kept>& kept() {
  static auto* m = new std::map<std::pair<int, uintptr_t>, Kept>();
  return *m;
}
std::vector<Kept>& retired() {
  static auto* v = new std::vector<Kept>();
  return *v;
}

RunResult workspace_of(const Clip& clip, size_t need, hipStream_t st, std::unique_lock<std::mutex>& lk, char** out) {
  RunResult r;
  if (clip.workspace) {
    if (clip.workspace_bytes < need) {
      r.status = 3;
      r.message = "workspace too small: need " + std::to_string(need) + " bytes";
      return r;
    }
    *out = static_cast<char*>(clip.workspace);
    return r;
  }
  // a captured call is replayed whenever its graph is, beside whatever else then uses this stream's
  // workspace: it has to bring one of its own
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  hipError_t e = hipStreamIsCapturing(st, &cs);
  if (e != hipSuccess) return hip_fail(e, "hipStreamIsCapturing");
  if (cs != hipStreamCaptureStatusNone) {
    r.status = 2;
    r.message = "a captured call needs a workspace of its own (" + std::to_string(need) + " bytes)";
    return r;
  }
  int device = 0;
  e = hipGetDevice(&device);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  lk = std::unique_lock<std::mutex>(g_mu);
  Kept& w = kept()[{device, reinterpret_cast<uintptr_t>(st)}];
  if (w.bytes < need) {
    void* p = nullptr;
    e = hipMalloc(&p, need);
    if (e != hipSuccess) return hip_fail(e, "allocating the workspace");
    if (w.p) retired().push_back(w);  // earlier launches on this stream may still use it
    w = Kept{p, need, device};
  }
  *out = static_cast<char*>(w.p);
  return r;
}

// The call's launches in order: the first records the start event, the last the stop event.
struct Sequence {
  hipStream_t st;
  Evs ev;
  int64_t left;
  bool begun = false;
  hipError_t err = hipSuccess;
  template <typename K, typename... A> void launch(K k, int64_t blocks, int threads, A... a) {
    if (err != hipSuccess) return;
    --left;
    hipExtLaunchKernelGGL(k, dim3(unsigned(blocks)), dim3(unsigned(threads)), 0, st, begun ? nullptr : ev.start,
                          left ? nullptr : ev.stop, 0, a...);
    begun = true;
    err = hipGetLastError();
  }
  RunResult done() {
    if (err == hipSuccess && !begun) {  // no launch: both events mark this point of the stream
      if (ev.start) err = hipEventRecord(ev.start, st);
      if (err == hipSuccess && ev.stop) err = hipEventRecord(ev.stop, st);
    }
    return err == hipSuccess ? RunResult{} : hip_fail(err, "launching the gradient kernels");
  }
};

int64_t blocks_for(int64_t items) { return std::max<int64_t>(1, std::min<int64_t>(items, launch_blocks())); }

#define AR_KIND(kind, ...)                                   \
  if ((kind) == N_L2) { constexpr int KIND = N_L2; __VA_ARGS__; } \
  else { constexpr int KIND = N_MAX; __VA_ARGS__; }

// Every tensor's or bucket's own norm from the call's partials.
void launch_each(Sequence& s, const Clip& clip, const std::vector<int32_t>& firsts, const double* partial) {
  const int64_t count = int64_t(firsts.size()) - 1;
  for (int64_t i0 = 0; i0 < count; i0 += kEachTensors) {
    EachTab tab;
    const int64_t c = std::min<int64_t>(kEachTensors, count - i0);
    std::memcpy(tab.first, firsts.data() + i0, size_t(c + 1) * sizeof(int32_t));
    AR_KIND(clip.norm, s.launch(k_norm_each<KIND>, c, 64, tab, partial, clip.each + i0));
  }
}

int64_t total_of(const Grad* g, int64_t count) {
  int64_t t = 0;
  for (int64_t i = 0; i < count; ++i) t += g[i].n;
  return t;
}

}  // namespace

size_t grad_workspace(const Grad* g, int64_t count, const Clip& clip) {
  if (clip.known) return 0;
  const int64_t per = item_size(total_of(g, count));
  int64_t items = 0;
  for (int64_t i = 0; i < count; ++i) items += pieces(g[i].n, per);
  return kHead + round_up(size_t(items) * sizeof(double));
}

RunResult run_grad(const Grad* g, int64_t count, const Clip& clip, bool scale, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t per = item_size(total_of(g, count));
  std::vector<GradTab> tabs;
  std::vector<int32_t> firsts{0};
  for (int64_t i0 = 0; i0 < count; i0 += kTabTensors) {
    GradTab tab;
    std::memset(&tab, 0, sizeof(tab));
    tab.count = int32_t(std::min<int64_t>(kTabTensors, count - i0));
    tab.at = firsts.back();
    tab.per = per;
    for (int k = 0; k < tab.count; ++k) {
      const Grad& t = g[i0 + k];
      tab.src[k] = t.data;
      tab.dst[k] = t.out;
      tab.n4[k] = (t.n << 2) | (t.out_dtype == D_BF16 ? 2 : 0) | (t.dtype == D_BF16 ? 1 : 0);
      tab.first[k + 1] = tab.first[k] + int32_t(pieces(t.n, per));
      firsts.push_back(tab.at + tab.first[k + 1]);
    }
    if (tab.first[tab.count]) tabs.push_back(tab);
  }
  const int32_t items = firsts.back();
  std::unique_lock<std::mutex> lk;
  char* ws = nullptr;
  if (!clip.known) {
    const RunResult r = workspace_of(clip, grad_workspace(g, count, clip), st, lk, &ws);
    if (r.status) return r;
  }
  double* norm = reinterpret_cast<double*>(ws);
  double* partial = reinterpret_cast<double*>(ws + kHead);
  Sequence s{st, {reinterpret_cast<hipEvent_t>(clip.start_event), reinterpret_cast<hipEvent_t>(clip.stop_event)}, 0};
  const int64_t nt = int64_t(tabs.size());
  s.left = (clip.known ? 0 : nt + 1 + (clip.each ? pieces(count, kEachTensors) : 0)) + (scale ? nt : 0);
  if (!clip.known) {
    for (const GradTab& t : tabs)
      AR_KIND(clip.norm, s.launch(k_grad_norm<KIND>, blocks_for(t.first[t.count]), kThreads, t, partial));
    AR_KIND(clip.norm, s.launch(k_norm_final<KIND>, 1, kFinalThreads, (const double*)partial, int(items), norm, clip.total));
    if (clip.each) launch_each(s, clip, firsts, partial);
  }
  if (scale)
    for (const GradTab& t : tabs)
      s.launch(k_grad_scale, blocks_for(t.first[t.count]), kThreads, t, (const double*)norm, clip.known, clip.max_norm,
               clip.eps);
  return s.done();
}

namespace {

template <int DT, int KIND> void launch_reduce(Sequence& s, int batch, int64_t blocks, const BucketTab& t, double* partial) {
#define AR_REDUCE(B_) s.launch(k_bucket_reduce<DT, KIND, B_>, blocks, kThreads, t, partial)
  switch (batch) {
    case 1: AR_REDUCE(1); break;
    case 2: AR_REDUCE(2); break;
    case 3: AR_REDUCE(3); break;
    case 4: AR_REDUCE(4); break;
    case 5: AR_REDUCE(5); break;
    case 6: AR_REDUCE(6); break;
    case 7: AR_REDUCE(7); break;
    default: AR_REDUCE(8); break;
  }
#undef AR_REDUCE
}

struct BucketPlan {
  std::vector<BucketTab> tabs;
  std::vector<int32_t> firsts{0};
  size_t low_bytes = 0;  // lower halves kept in the workspace
};

bool low_in_workspace(const Buckets& b) { return b.dtype == D_BF16 && b.coll == C_REDUCE_SCATTER && b.P > 1; }

BucketPlan plan_buckets(const Buckets& b) {
  BucketPlan pl;
  int64_t total = 0;
  for (int64_t i = 0; i < b.count; ++i) total += b.n[i];
  const int64_t per = item_size(total), fit = std::min<int64_t>(kTabBuckets, kTabPtrs / b.P);
  const bool scatter = b.coll == C_REDUCE_SCATTER;
  for (int64_t i0 = 0; i0 < b.count; i0 += fit) {
    BucketTab tab;
    std::memset(&tab, 0, sizeof(tab));
    tab.count = int32_t(std::min(fit, b.count - i0));
    tab.P = b.P;
    tab.at = pl.firsts.back();
    tab.owners = scatter;
    tab.per = per;
    tab.div = b.op == O_AVG ? float(b.P) : 0.0f;
    for (int k = 0; k < tab.count; ++k) {
      const int64_t n = b.n[i0 + k], part = scatter ? pieces(n, b.P) : n;
      for (int q = 0; q < b.P; ++q) tab.p[k * b.P + q] = b.bufs ? b.bufs[(i0 + k) * b.P + q] : nullptr;  // none: only the size is asked
      tab.n[k] = n;
      tab.part[k] = part;
      tab.ipp[k] = int32_t(std::max<int64_t>(1, pieces(part, per)));
      if (low_in_workspace(b)) {
        tab.low[k] = reinterpret_cast<uint16_t*>(pl.low_bytes);  // an offset until the workspace is known
        pl.low_bytes += round_up(size_t(n) * 2);
      } else if (b.dtype == D_BF16 && b.P > 1) {
        tab.low[k] = static_cast<uint16_t*>(tab.p[k * b.P + 1]);
      }
      tab.first[k + 1] = tab.first[k] + (n ? tab.ipp[k] * (scatter ? b.P : 1) : 0);
      pl.firsts.push_back(tab.at + tab.first[k + 1]);
    }
    if (tab.first[tab.count]) pl.tabs.push_back(tab);
  }
  return pl;
}

size_t bucket_bytes(const BucketPlan& pl) { return kHead + round_up(size_t(pl.firsts.back()) * sizeof(double)) + pl.low_bytes; }

}  // namespace

size_t allreduce_clip_workspace(const Buckets& b, const Clip&) { return bucket_bytes(plan_buckets(b)); }

RunResult run_allreduce_clip(const Buckets& b, const Clip& clip, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  BucketPlan pl = plan_buckets(b);
  std::unique_lock<std::mutex> lk;
  char* ws = nullptr;
  const RunResult r = workspace_of(clip, bucket_bytes(pl), st, lk, &ws);
  if (r.status) return r;
  double* norm = reinterpret_cast<double*>(ws);
  double* partial = reinterpret_cast<double*>(ws + kHead);
  if (low_in_workspace(b)) {
    char* low = ws + kHead + round_up(size_t(pl.firsts.back()) * sizeof(double));
    for (BucketTab& t : pl.tabs)
      for (int k = 0; k < t.count; ++k) t.low[k] = reinterpret_cast<uint16_t*>(low + reinterpret_cast<size_t>(t.low[k]));
  }
  Sequence s{st, {reinterpret_cast<hipEvent_t>(clip.start_event), reinterpret_cast<hipEvent_t>(clip.stop_event)}, 0};
  s.left = 2 * int64_t(pl.tabs.size()) + 1 + (clip.each ? pieces(b.count, kEachTensors) : 0);
  for (const BucketTab& t : pl.tabs) {
    const int64_t blocks = blocks_for(t.first[t.count]);
    if (b.dtype == D_BF16) { AR_KIND(clip.norm, launch_reduce<D_BF16, KIND>(s, leaf_batch(b.P), blocks, t, partial)); }
    else { AR_KIND(clip.norm, launch_reduce<D_FP32, KIND>(s, leaf_batch(b.P), blocks, t, partial)); }
  }
  AR_KIND(clip.norm, s.launch(k_norm_final<KIND>, 1, kFinalThreads, (const double*)partial, int(pl.firsts.back()), norm, clip.total));
  if (clip.each) launch_each(s, clip, pl.firsts, partial);
  for (const BucketTab& t : pl.tabs) {
    const int64_t blocks = blocks_for(t.first[t.count]);
    if (b.dtype == D_BF16) s.launch(k_bucket_spread<D_BF16>, blocks, kThreads, t, (const double*)norm, clip.max_norm, clip.eps);
    else s.launch(k_bucket_spread<D_FP32>, blocks, kThreads, t, (const double*)norm, clip.max_norm, clip.eps);
  }
  return s.done();
}

GradCache grad_cache() {
  std::lock_guard<std::mutex> lk(g_mu);
  GradCache c;
  for (const auto& kv : kept()) {
    if (kv.second.p) ++c.live;
    c.bytes += int64_t(kv.second.bytes);
  }
  for (const Kept& w : retired()) {
    ++c.retired;
    c.bytes += int64_t(w.bytes);
  }
  return c;
}

void grad_cache_devices(void (*note)(int, void*), void* to) {
  std::lock_guard<std::mutex> lk(g_mu);
  for (const auto& kv : kept()) note(kv.first.first, to);
  for (const Kept& w : retired()) note(w.device, to);
}

void grad_cache_free() {
  std::lock_guard<std::mutex> lk(g_mu);
  for (auto& kv : kept())
    if (kv.second.p) (void)hipFree(kv.second.p);
  for (Kept& w : retired()) (void)hipFree(w.p);
  kept().clear();
  retired().clear();
}

}  // namespace ar
