// Gradient norms and clipping for gfx950: the global norm over many tensors, the
// scaling that limits it, and both inside the Allreduce of P rank buffers.
//
//   N     = sqrt(sum over every element of g^2), or the largest |g|
//   scale = 1 where N + eps <= max_norm, else max_norm / (N + eps)
//   y     = scale g
//
// Every pass streams memory; the arithmetic per element is a widening, a
// multiply-add in 64 bits and one multiplication. Tensors are cut into work items
// of `per` elements, which a launch's workgroups take in turn; each leaves one
// partial norm at its own place, and whoever needs the norm joins the partials in
// their order. Nothing is added atomically: the same sizes, device and launch limit
// give the same bits, whatever runs beside the call and wherever the tensors lie.
//
// The scale is rounded from 64 bits to fp32, its product with g to fp32, and a bf16 y from that: each
// element costs one fp32 multiplication (2^-23 in all, and 2^-8 more in bf16). A product in 64 bits would
// save the middle rounding, a 2^-16th of bf16's own.
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
#include <set>
#include <vector>

#include "kernels.h"
#include "sequence.h"

namespace ar {

// ----------------------------------------------------------------------------
// arithmetic
// ----------------------------------------------------------------------------
// Vectors of 16 bytes at any element's address: global accesses of this target
// need no alignment, and a tensor's vectors are counted from its first element, so
// how it is cut (and the order of its sums) does not depend on where it lies.
template <int DT, int V> struct Raw;
template <> struct Raw<D_FP32, 4> { typedef uint32_t T __attribute__((ext_vector_type(4), aligned(4))); };
template <> struct Raw<D_BF16, 8> { typedef uint32_t T __attribute__((ext_vector_type(4), aligned(2))); };
template <> struct Raw<D_BF16, 4> { typedef uint32_t T __attribute__((ext_vector_type(2), aligned(2))); };

// fp32 -> bf16 bits, to nearest even; NaN stays NaN (a carry out of a NaN's
// payload would make it an infinity or a zero).
__device__ __forceinline__ uint32_t bf16_of(float f) {
  const uint32_t u = as_u(f);
  const uint32_t r = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
  return (u & 0x7fffffffu) > 0x7f800000u ? (u >> 16) | 0x40u : r;
}

// V elements as they lie in memory, and their values. NT: with the non-temporal hint.
template <int DT, int V, bool NT> __device__ __forceinline__ typename Raw<DT, V>::T ld_raw(const void* base, int64_t e) {
  const auto* p = reinterpret_cast<const typename Raw<DT, V>::T*>(static_cast<const typename TT<DT>::S*>(base) + e);
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}

template <int DT, int V, bool NT> __device__ __forceinline__ void st_raw(void* base, int64_t e, typename Raw<DT, V>::T r) {
  auto* p = reinterpret_cast<typename Raw<DT, V>::T*>(static_cast<typename TT<DT>::S*>(base) + e);
  if constexpr (NT) __builtin_nontemporal_store(r, p);
  else *p = r;
}

template <int DT, int V> __device__ __forceinline__ float value(const typename Raw<DT, V>::T& r, int i) {
  if constexpr (DT == D_FP32) return as_f(r[i]);
  else return as_f(i % 2 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
}

template <int DT, int V> __device__ __forceinline__ typename Raw<DT, V>::T pack(const float (&x)[V]) {
  typename Raw<DT, V>::T r;
  if constexpr (DT == D_FP32) {
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = as_u(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r[i] = bf16_of(x[2 * i]) | (bf16_of(x[2 * i + 1]) << 16);
  }
  return r;
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

// What a thread gathers over an item's elements: squares in 64 bits, or magnitudes as fp32 patterns, one
// operation an element.
template <int KIND> struct Gather;
template <> struct Gather<N_L2> {
  double v = 0;
  __device__ __forceinline__ void add(float x) {
    const double d = double(x);
    v = __builtin_fma(d, d, v);
  }
  __device__ __forceinline__ double value() const { return v; }
};
template <> struct Gather<N_MAX> {
  uint32_t m = 0;
  __device__ __forceinline__ void add(float x) { m = max(m, as_u(x) & 0x7fffffffu); }
  __device__ __forceinline__ double value() const { return double(as_f(m)); }
};

template <int KIND> __device__ __forceinline__ void join_wave(Part<KIND>& p) {  // valid in lane 0
#pragma unroll
  for (int d = 32; d; d >>= 1) p.join(__shfl_down(p.v, d));
}

// The workgroup's partial, valid in thread 0: within a wave by shuffles, then over the waves in order.
template <int KIND, int THREADS> __device__ __forceinline__ void join_group(Part<KIND>& p) {
  __shared__ double wave[THREADS / 64];
  join_wave(p);
  __syncthreads();  // the array's last readers
  if (threadIdx.x % 64 == 0) wave[threadIdx.x / 64] = p.v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < THREADS / 64; ++w) p.join(wave[w]);
}

// An item's partials, one from each wave: its workgroup need not meet.
constexpr int kWaves = kThreads / 64;
template <int KIND> __device__ __forceinline__ void put_waves(Part<KIND> p, double* partial) {
  join_wave(p);
  if (threadIdx.x % 64 == 0) partial[threadIdx.x / 64] = p.v;
}

// `count` partials joined in one order, the result in thread 0: a thread's loads are in flight together.
template <int KIND, int THREADS> __device__ __forceinline__ Part<KIND> join_partials(const double* partial, int count) {
  constexpr int U = 8;
  Part<KIND> p;
  for (int i = threadIdx.x; i < count; i += U * THREADS) {
    double x[U];
#pragma unroll
    for (int j = 0; j < U; ++j) x[j] = i + j * THREADS < count ? partial[i + j * THREADS] : 0.0;
#pragma unroll
    for (int j = 0; j < U; ++j) p.join(x[j]);
  }
  join_group<KIND, THREADS>(p);
  return p;
}

// The norm that a call's partials make, in every thread of a workgroup: each of them joins them by
// itself, which costs less than a launch between two passes.
template <int KIND, int THREADS> __device__ __forceinline__ Part<KIND> join_all(const double* partial, int count) {
  __shared__ double all;
  Part<KIND> p = join_partials<KIND, THREADS>(partial, count);
  if (threadIdx.x == 0) all = p.v;
  __syncthreads();
  p.v = all;
  return p;
}

// The scale as a product a b of two fp32 values: one where it has fp32's full precision, and below
// 2^-64 (a limit far under an exploding norm) two halves of its exponent, so that x a b is right for
// every x and rounds once more only where the result has no 24 bits. b stays at fp32's smallest value where
// its half of the exponent lies below (scales under 2^-274: a denormal limit and a norm near fp32's end), a takes
// the rest and keeps the few bits that a result there has; neither ever becomes zero, which would turn an
// infinity into NaN.
struct Factor {
  float a, b;
  __device__ __forceinline__ bool one() const { return a == 1.0f && b == 1.0f; }
  __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};

__device__ __forceinline__ Factor factor_of(double norm, float max_norm, float eps) {
  const double reach = norm + double(eps);
  const double s = reach <= double(max_norm) ? 1.0 : double(max_norm) / reach;  // a NaN stays one
  if (s > 0 && s < 0x1p-64) {
    int e;
    const double m = frexp(s, &e);
    const int eb = max(e - max(e / 2, -125), -149);
    return {float(fmax(ldexp(m, e - eb), 0x1p-149)), float(ldexp(1.0, eb))};
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
  int32_t at;     // place of this launch's first partial among the call's
  int32_t item0;  // its first item among the call's
  int64_t per;    // elements per work item
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

// L lanes (a workgroup's, or a wave's), of which this is `lane`, go over an item together.
template <int KIND, int DT, int L, bool NT> __device__ __forceinline__ void norm_item(const void* src, int64_t e0, int cnt, int lane, Gather<KIND>& p) {
  constexpr int V = DT == D_BF16 ? 8 : 4;
  constexpr int U = L == 64 ? 4 : 2;  // vectors of a thread in flight; with 24 waves on a compute unit two do (990 M bf16: 303 us of 4, 298 of 2)
  const int nv = cnt / V;
  int v = lane;
  for (; v + (U - 1) * L < nv; v += U * L) {
    typename Raw<DT, V>::T r[U];
#pragma unroll
    for (int j = 0; j < U; ++j) r[j] = ld_raw<DT, V, NT>(src, e0 + int64_t(v + j * L) * V);
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) p.add(value<DT, V>(r[j], i));
  }
  for (; v < nv; v += L) {
    const typename Raw<DT, V>::T r = ld_raw<DT, V, NT>(src, e0 + int64_t(v) * V);
#pragma unroll
    for (int i = 0; i < V; ++i) p.add(value<DT, V>(r, i));
  }
  const int t = nv * V + lane;
  if (t < cnt) p.add(ld_one<DT>(src, e0 + t));
}

// One item of a list: its tensor, first element and elements (at most `per`, which fits an int).
struct GradItem {
  int i;
  int64_t e0;
  int cnt;
};
__device__ __forceinline__ GradItem grad_item(const GradTab& tab, int it) {
  GradItem w;
  w.i = find_first(tab, tab.count, it);
  w.e0 = int64_t(it - tab.first[w.i]) * tab.per;
  w.cnt = int(min(tab.per, (tab.n4[w.i] >> 2) - w.e0));
  return w;
}

// A partial for every workgroup over all of its items, and (EACH) `own` ones for every item, which the
// tensors' norms are joined from. NT (a norm alone, and every EACH): the loads leave the cache in front of HBM
// to others, 990 M bf16 355 -> 326 us; a pass that a scaling follows leaves its last part there. A clip that
// asks for the tensors' own norms too has no such form: its passes over 187 M bf16 into bf16 take 58, 5 and
// 137 us, without own norms 63 and 112.
//
// Bound by HBM reads: 234 us for 1.58 GB of bf16, 6.7 TB/s; 25 us for 143 MB of ragged fp32, 5.6 TB/s. 24
// waves to a compute unit cover the latency.
template <int KIND, bool EACH, bool NT> __global__ __launch_bounds__(kThreads) void k_grad_norm(GradTab tab, double* partial, double* own) {
  Part<KIND> all;
  Gather<KIND> p;
  for (int it = blockIdx.x; it < tab.first[tab.count]; it += gridDim.x) {
    const GradItem w = grad_item(tab, it);
    if (tab.n4[w.i] & 1) norm_item<KIND, D_BF16, kThreads, NT>(tab.src[w.i], w.e0, w.cnt, threadIdx.x, p);
    else norm_item<KIND, D_FP32, kThreads, NT>(tab.src[w.i], w.e0, w.cnt, threadIdx.x, p);
    if constexpr (EACH) {
      all.join(p.value());
      put_waves(Part<KIND>{p.value()}, own + int64_t(tab.item0 + it) * kWaves);
      p = Gather<KIND>();
    }
  }
  if constexpr (!EACH) all.v = p.value();
  join_group<KIND, kThreads>(all);
  if (threadIdx.x == 0) partial[tab.at + blockIdx.x] = all.v;
}

// The tensors' own norms, a workgroup to a tensor, and behind the last tensor the call's. `joined` is for a
// pass that scales. 4-5 us, most of them a launch's own.
constexpr int kFinalThreads = 512, kEachTensors = 900;
struct EachTab {
  int32_t first[kEachTensors + 1];  // first partial of every tensor
  int32_t count;
};

template <int KIND> __global__ __launch_bounds__(kFinalThreads) void k_norm_final(EachTab tab, const double* partial, int count, const double* own, double* joined, float* total, float* each) {
  const int i = blockIdx.x;
  if (i < tab.count) {
    const Part<KIND> p = join_partials<KIND, kFinalThreads>(own + tab.first[i], tab.first[i + 1] - tab.first[i]);
    if (threadIdx.x == 0) each[i] = float(p.norm());
  } else {
    const Part<KIND> p = join_partials<KIND, kFinalThreads>(partial, count);
    if (threadIdx.x == 0) {
      *joined = p.v;
      if (total) *total = float(p.norm());
    }
  }
}

template <int DS, int DD, int L> __device__ __forceinline__ void scale_item(const void* src, void* dst, int64_t e0, int cnt, int lane, Factor f) {
  // between the types, 4 elements a thread: its stores (or loads) then join its neighbours' to whole lines
  constexpr int V = DS == D_BF16 && DD == D_BF16 ? 8 : 4;
  constexpr int U = 64 / sizeof(typename Raw<DS, V>::T);  // 64 bytes of a thread in flight (bf16 into fp32, 477 M: 671 us of 32 bytes, 658 of 64)
  const int nv = cnt / V;
  int v = lane;
  for (; v + (U - 1) * L < nv; v += U * L) {
    typename Raw<DS, V>::T r[U];
#pragma unroll
    for (int j = 0; j < U; ++j) r[j] = ld_raw<DS, V, true>(src, e0 + int64_t(v + j * L) * V);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float x[V];
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = f(value<DS, V>(r[j], i));
      st_raw<DD, V, true>(dst, e0 + int64_t(v + j * L) * V, pack<DD, V>(x));
    }
  }
  for (; v < nv; v += L) {
    const typename Raw<DS, V>::T r = ld_raw<DS, V, true>(src, e0 + int64_t(v) * V);
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = f(value<DS, V>(r, i));
    st_raw<DD, V, true>(dst, e0 + int64_t(v) * V, pack<DD, V>(x));
  }
  const int t = nv * V + lane;
  if (t < cnt) st_one<DD>(dst, e0 + t, f(ld_one<DS>(src, e0 + t)));
}

template <int L> __device__ __forceinline__ void scale_any(const GradTab& tab, const GradItem& w, int lane, Factor f) {
  const void* s = tab.src[w.i];
  void* d = tab.dst[w.i];
  if (f.one() && s == d) return;  // within the limit and in place: the gradient is its own result
  switch (int(tab.n4[w.i] & 3)) {
    case 0: scale_item<D_FP32, D_FP32, L>(s, d, w.e0, w.cnt, lane, f); break;
    case 1: scale_item<D_BF16, D_FP32, L>(s, d, w.e0, w.cnt, lane, f); break;
    case 2: scale_item<D_FP32, D_BF16, L>(s, d, w.e0, w.cnt, lane, f); break;
    default: scale_item<D_BF16, D_BF16, L>(s, d, w.e0, w.cnt, lane, f); break;
  }
}

// What the passes that scale start from.
struct Limit {
  const double* partial;
  int32_t count;
  float max_norm, eps;
  const float* known;  // instead of partials
  float* total;        // written by the call's first such launch, or null
  bool in_place;       // a list whose tensors all stay where they are: within the limit nothing is to be done
};

template <int KIND> __device__ __forceinline__ Factor factor_for(const Limit& lim) {
  if (lim.known) return factor_of(double(*lim.known), lim.max_norm, lim.eps);
  const double norm = join_all<KIND, kThreads>(lim.partial, lim.count).norm();
  if (lim.total && blockIdx.x == 0 && threadIdx.x == 0) *lim.total = float(norm);
  return factor_of(norm, lim.max_norm, lim.eps);
}

// The last item of a workgroup's share of `items`. The scaling pass begins there and goes backwards: what
// the norm read last is still in the cache in front of HBM (256 MB), and neither the loads here nor the
// stores displace it. Norm and scaling of 187 M bf16 into bf16: 242 us forwards with plain accesses, 205
// with non-temporal ones, 193 backwards too (175 with 64 bytes in flight); 187 M fp32: 452, 376, 375.
__device__ __forceinline__ int last_item(int items) { return items - 1 - int((items - 1 - blockIdx.x) % gridDim.x); }

// Bound by HBM, reads and writes together: 501 us for 477 M bf16 into fp32 (2.86 GB, 5.7 TB/s), 280 us for
// 187 M fp32 in place (1.50 GB, 5.4 TB/s); in place within the limit there is nothing to write, and the
// clip of 187 M fp32 takes 129 us, 124 of them the norm's.
template <int KIND> __global__ __launch_bounds__(kThreads) void k_grad_scale(GradTab tab, Limit lim) {
  const Factor f = factor_for<KIND>(lim);
  if (lim.in_place && f.one()) return;
  for (int k = last_item(tab.first[tab.count]); k >= 0; k -= int(gridDim.x)) scale_any<kThreads>(tab, grad_item(tab, k), threadIdx.x, f);
}

// A short list in one launch: one workgroup, whose waves take an item each. Its second look at the
// elements finds them in the L2. Bound by what one compute unit takes in: 5.0 us for the norm of 63 k fp32
// elements, 6.3 for the clip of 12 tensors of 2048.
constexpr int kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64, kSmallItems = 48;
template <int KIND, bool SCALE>
__global__ __launch_bounds__(kSmallThreads) void k_grad_small(GradTab tab, float* total, float* each, float max_norm, float eps) {
  __shared__ double own[kSmallItems];
  __shared__ double all;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, items = tab.first[tab.count];
  Part<KIND> p;
  for (int it = wave; it < items; it += kSmallWaves) {
    const GradItem w = grad_item(tab, it);
    Gather<KIND> g;
    if (tab.n4[w.i] & 1) norm_item<KIND, D_BF16, 64, false>(tab.src[w.i], w.e0, w.cnt, lane, g);
    else norm_item<KIND, D_FP32, 64, false>(tab.src[w.i], w.e0, w.cnt, lane, g);
    Part<KIND> q{g.value()};
    p.join(q.v);
    if (each) {
      join_wave(q);
      if (lane == 0) own[it] = q.v;
    }
  }
  join_group<KIND, kSmallThreads>(p);
  if (threadIdx.x == 0) {
    all = p.norm();
    if (total) *total = float(all);
  }
  __syncthreads();
  if (each)
    for (int i = threadIdx.x; i < tab.count; i += kSmallThreads) {
      Part<KIND> q;
      for (int k = tab.first[i]; k < tab.first[i + 1]; ++k) q.join(own[k]);
      each[i] = float(q.norm());
    }
  if constexpr (SCALE) {
    const Factor f = factor_of(all, max_norm, eps);
    for (int it = wave; it < items; it += kSmallWaves) scale_any<64>(tab, grad_item(tab, it), lane, f);
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
// Few ranks are read twice instead, and no sum is kept: the Allreduce then moves 3 P elements in place of
// 2 P + 2 in fp32, and of 2 P + 4 in bf16, whose fp32 sums take two each.
// A bucket's pointers fill whole batches of kRankBatch, the last one again behind the last rank: a
// batch's pointers are then one scalar load, and its ranks' loads go out together with no test between
// them. Most of the repeated loads find their lines in the cache, not all: of 400 MB of fp32, 9 ranks read
// 444 (93 us, where 8 ranks take 79), 17 ranks 421 (83, 16 take 76) and 33 ranks 409 (75, 32 take 71).
constexpr int kTabPtrs = 400, kTabBuckets = 16, kRankBatch = 16;
struct BucketTab {
  void* p[kTabPtrs];               // `stride` pointers of every bucket
  uint16_t* low[kTabBuckets];      // lower halves of bf16 sums, by element
  int64_t part[kTabBuckets];       // elements per part (the whole bucket for the Allreduce)
  int64_t n[kTabBuckets];
  int32_t first[kTabBuckets + 1];  // first work item
  int32_t ipp[kTabBuckets];        // work items per part
  int32_t count, P, stride;
  int32_t at, item0;               // as in GradTab
  int32_t owners;                  // 1: part q belongs to rank q alone
  int64_t per;
  float div;                       // > 0: the sum is divided by it
};
static_assert(sizeof(BucketTab) <= 4000, "kernel arguments");

struct BucketItem {
  int b, owner;
  int64_t e0;
  int cnt;
};

__device__ __forceinline__ BucketItem bucket_item(const BucketTab& tab, int it) {
  BucketItem r;
  r.b = find_first(tab, tab.count, it);
  const int k = it - tab.first[r.b], q = k / tab.ipp[r.b];
  r.owner = tab.owners ? q : 0;
  const int64_t lo = q * tab.part[r.b], hi = min(lo + tab.part[r.b], tab.n[r.b]);
  r.e0 = lo + (k - q * tab.ipp[r.b]) * tab.per;
  r.cnt = int(max(int64_t(0), min(tab.per, hi - r.e0)));  // the last parts may be short or empty
  return r;
}

// The ranks' vectors are read once, in batches of B ranks whose loads are all in flight before the first
// is added; a thread's M vectors go together. One load at a time took 135 us for the sums of 7 x 2^24
// fp32 and 134 us for those of 192 x 2^20 bf16, a batch 92 and 64; loading the next batch before adding
// this one gained nothing (178 and 132 us for the whole call, against 175 and 135).
template <int DT, int V, int M, int B, bool NT>
__device__ __forceinline__ void ld_ranks(void* const* ptr, int base, int64_t e, const bool (&ok)[M], typename Raw<DT, V>::T (&r)[B][M]) {
#pragma unroll
  for (int k = 0; k < B; ++k) {
    const void* p = ptr[base + k];
#pragma unroll
    for (int j = 0; j < M; ++j)
      if (ok[j]) r[k][j] = ld_raw<DT, V, NT>(p, e + j * kThreads * V);
  }
}

template <int DT, int V, int M, int B>
__device__ __forceinline__ void add_ranks(int P, int base, const typename Raw<DT, V>::T (&r)[B][M], float (&acc)[M][V]) {
#pragma unroll
  for (int k = 0; k < B; ++k) {
    if (base + k >= P) continue;
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float x = value<DT, V>(r[k][j], i);
        acc[j][i] = base + k ? acc[j][i] + x : x;
      }
  }
}

template <int DT, int V, int M, int B, bool NT>
__device__ __forceinline__ void sum_ranks(void* const* ptr, int P, float div, int64_t e, const bool (&ok)[M], float (&acc)[M][V]) {
  for (int base = 0; base < P; base += B) {
    typename Raw<DT, V>::T r[B][M];
    ld_ranks<DT, V, M, B, NT>(ptr, base, e, ok, r);
    add_ranks<DT, V, M, B>(P, base, r, acc);
  }
  if (div > 0) {
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[j][i] = acc[j][i] / div;
  }
}

// One element's sum: what lies behind the last whole vector has as many ranks to wait for as the rest.
template <int DT> __device__ __forceinline__ float sum_one(void* const* ptr, int P, float div, int64_t e) {
  float acc = 0;
  for (int base = 0; base < P; base += kRankBatch) {
    float x[kRankBatch];
#pragma unroll
    for (int r = 0; r < kRankBatch; ++r) x[r] = ld_one<DT>(ptr[base + r], e);
#pragma unroll
    for (int r = 0; r < kRankBatch; ++r)
      if (base + r < P) acc = base + r ? acc + x[r] : x[r];
  }
  return div > 0 ? acc / div : acc;
}

// f(rank's buffer) for ranks [q0, q1), with their pointers looked up together.
template <typename F> __device__ __forceinline__ void to_ranks(void* const* ptr, int q0, int q1, F&& f) {
  int q = q0;
  for (; q + 8 <= q1; q += 8) {
    void* p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = ptr[q + k];
#pragma unroll
    for (int k = 0; k < 8; ++k) f(p[k]);
  }
  for (; q < q1; ++q) f(ptr[q]);
}

// Whole sums to and from their place.
template <int DT, int V> __device__ __forceinline__ void put_sum(void* own, uint16_t* low, int64_t e, const float (&s)[V]) {
  if constexpr (DT == D_FP32) {
    st_raw<D_FP32, V, false>(own, e, pack<D_FP32, V>(s));
  } else {
    typename Raw<D_BF16, V>::T h, l;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const uint32_t a = as_u(s[2 * i]), b = as_u(s[2 * i + 1]);
      h[i] = (a >> 16) | (b & 0xffff0000u);
      l[i] = (a & 0xffffu) | (b << 16);
    }
    st_raw<D_BF16, V, false>(own, e, h);
    st_raw<D_BF16, V, false>(low, e, l);
  }
}

template <int DT> __device__ __forceinline__ void put_one(void* own, uint16_t* low, int64_t e, float s) {
  if constexpr (DT == D_FP32) {
    static_cast<float*>(own)[e] = s;
  } else {
    static_cast<uint16_t*>(own)[e] = uint16_t(as_u(s) >> 16);
    low[e] = uint16_t(as_u(s));
  }
}

template <int DT, int V> __device__ __forceinline__ void get_sum(const void* own, const uint16_t* low, int64_t e, float (&s)[V]) {
  const typename Raw<DT, V>::T h = ld_raw<DT, V, false>(own, e);
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = value<DT, V>(h, i);
  if constexpr (DT == D_BF16) {
    const typename Raw<DT, V>::T l = ld_raw<DT, V, false>(low, e);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = as_f(as_u(s[i]) | (i % 2 ? l[i / 2] >> 16 : l[i / 2] & 0xffffu));
  }
}

template <int DT> __device__ __forceinline__ float get_one(const void* own, const uint16_t* low, int64_t e) {
  const float s = ld_one<DT>(own, e);
  return DT == D_BF16 ? as_f(as_u(s) | low[e]) : s;
}

// Vectors of a thread that go together: an item of 2048 elements is one for bf16 and two for fp32.
template <int DT> constexpr int kPair = DT == D_BF16 ? 1 : 2;

// The first pass. KEEP: the sums stay for the second one, which otherwise reads the ranks again. Bound by
// HBM: 7 x 2^24 fp32 92 us (470 MB read, 67 written, 5.8 TB/s), 192 x 2^20 bf16 64 us (403 and 4 MB,
// 6.3 TB/s), 8 x 4 x 25 MB bf16 into parts 194 us (839 and 210 MB, 5.4 TB/s); 8 x 2^20 fp32 9-11 us, one
// round of loads.
template <int DT, int KIND, int B, int M, bool EACH, bool KEEP>
__global__ __launch_bounds__(kThreads) void k_bucket_reduce(BucketTab tab, double* partial, double* own) {
  constexpr int V = DT == D_BF16 ? 8 : 4;
  Part<KIND> all;
  Gather<KIND> p;
  for (int it = blockIdx.x; it < tab.first[tab.count]; it += gridDim.x) {
    const BucketItem w = bucket_item(tab, it);
    void* const* ptr = tab.p + w.b * tab.stride;
    const int nv = w.cnt / V;
    for (int v = threadIdx.x; v < nv; v += kThreads * M) {
      bool ok[M];
#pragma unroll
      for (int j = 0; j < M; ++j) ok[j] = v + j * kThreads < nv;
      float s[M][V];
      sum_ranks<DT, V, M, B, KEEP>(ptr, tab.P, tab.div, w.e0 + int64_t(v) * V, ok, s);
#pragma unroll
      for (int j = 0; j < M; ++j)
        if (ok[j]) {
#pragma unroll
          for (int i = 0; i < V; ++i) p.add(s[j][i]);
          if constexpr (KEEP) put_sum<DT, V>(ptr[w.owner], tab.low[w.b], w.e0 + int64_t(v + j * kThreads) * V, s[j]);
        }
    }
    const int t = nv * V + threadIdx.x;
    if (t < w.cnt) {
      const float s = sum_one<DT>(ptr, tab.P, tab.div, w.e0 + t);
      p.add(s);
      if constexpr (KEEP) put_one<DT>(ptr[w.owner], tab.low[w.b], w.e0 + t, s);
    }
    if constexpr (EACH) {
      all.join(p.value());
      put_waves(Part<KIND>{p.value()}, own + int64_t(tab.item0 + it) * kWaves);
      p = Gather<KIND>();
    }
  }
  if constexpr (!EACH) all.v = p.value();
  join_group<KIND, kThreads>(all);
  if (threadIdx.x == 0) partial[tab.at + blockIdx.x] = all.v;
}

// Items go in the first pass's order, workgroup by workgroup: the sums are read on the XCD that wrote
// them, out of its L2 or the cache in front of HBM, which the stores to the ranks do not pass through
// (7 x 2^24 fp32: 213 us for the call with plain stores, 178 with these). Bound by HBM writes: 7 x 2^24
// 84 us, 6.4 TB/s; 192 x 2^20 bf16 73 us, 5.6 TB/s; parts of 4 x 25 MB 51 us, 6.1 TB/s.
//
// B > 0: the first pass kept no sums, and this one makes them again from B ranks, backwards from what the
// first read last.
template <int DT, int KIND, int B> __global__ __launch_bounds__(kThreads) void k_bucket_spread(BucketTab tab, Limit lim) {
  constexpr int V = DT == D_BF16 ? 8 : 4, M = kPair<DT>;
  const Factor f = factor_for<KIND>(lim);
  if (DT == D_FP32 && B == 0 && tab.owners && f.one()) return;  // the sums are in their owners' parts already
  const int items = tab.first[tab.count], step = B ? -int(gridDim.x) : int(gridDim.x);
  for (int it = B ? last_item(items) : blockIdx.x; B ? it >= 0 : it < items; it += step) {
    const BucketItem w = bucket_item(tab, it);
    void* const* ptr = tab.p + w.b * tab.stride;
    const int q0 = tab.owners ? w.owner : 0, q1 = tab.owners ? w.owner + 1 : tab.P;
    const int nv = w.cnt / V;
    for (int v = threadIdx.x; v < nv; v += kThreads * M) {
      const int64_t e = w.e0 + int64_t(v) * V;
      bool ok[M];
      float s[M][V];
#pragma unroll
      for (int j = 0; j < M; ++j) ok[j] = v + j * kThreads < nv;
      if constexpr (B > 0) {
        sum_ranks<DT, V, M, B, true>(ptr, tab.P, tab.div, e, ok, s);
      } else {
#pragma unroll
        for (int j = 0; j < M; ++j)
          if (ok[j]) get_sum<DT, V>(ptr[w.owner], tab.low[w.b], e + j * kThreads * V, s[j]);
      }
      typename Raw<DT, V>::T y[M];
#pragma unroll
      for (int j = 0; j < M; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[j][i] = f(s[j][i]);
        y[j] = pack<DT, V>(s[j]);
      }
      to_ranks(ptr, q0, q1, [&](void* p) {
#pragma unroll
        for (int j = 0; j < M; ++j)
          if (ok[j]) st_raw<DT, V, true>(p, e + j * kThreads * V, y[j]);
      });
    }
    const int t = nv * V + threadIdx.x;
    if (t < w.cnt) {
      const float s = f(B ? sum_one<DT>(ptr, tab.P, tab.div, w.e0 + t) : get_one<DT>(ptr[w.owner], tab.low[w.b], w.e0 + t));
      to_ranks(ptr, q0, q1, [&](void* p) { st_one<DT>(p, w.e0 + t, s); });
    }
  }
}

// Few elements in one launch: one workgroup, whose waves take an item of 64 elements each and keep their sums
// in registers between the passes (8 x 1024 fp32: 5.4 us against 6.7 for two launches, 24 x 106: 5.6 and
// 12.6; with two items to a wave, 8 x 2048, 8.3 and 6.9).
constexpr int kSmallSpan = 64;
template <int DT, int KIND>
__global__ __launch_bounds__(kSmallThreads) void k_bucket_small(BucketTab tab, float* total, float* each, float max_norm, float eps) {
  __shared__ double own[kSmallWaves];
  __shared__ double all;
  const int it = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  Part<KIND> p;
  BucketItem w{0, 0, 0, 0};
  float sum = 0;
  if (it < tab.first[tab.count]) w = bucket_item(tab, it);
  void* const* ptr = tab.p + w.b * tab.stride;
  if (lane < w.cnt) {
    sum = sum_one<DT>(ptr, tab.P, tab.div, w.e0 + lane);
    Gather<KIND> g;
    g.add(sum);
    p.v = g.value();
  }
  if (each) {
    Part<KIND> q = p;
    join_wave(q);
    if (lane == 0) own[it] = q.v;
  }
  join_group<KIND, kSmallThreads>(p);
  if (threadIdx.x == 0) {
    all = p.norm();
    if (total) *total = float(all);
  }
  __syncthreads();
  if (each && threadIdx.x < tab.count) {
    Part<KIND> q;
    for (int k = tab.first[threadIdx.x]; k < tab.first[threadIdx.x + 1]; ++k) q.join(own[k]);
    each[threadIdx.x] = float(q.norm());
  }
  const float y = factor_of(all, max_norm, eps)(sum);
  const int q0 = tab.owners ? w.owner : 0, q1 = tab.owners ? w.owner + 1 : tab.P;
  if (lane < w.cnt) to_ranks(ptr, q0, q1, [&](void* p) { st_one<DT>(p, w.e0 + lane, y); });
}

// ----------------------------------------------------------------------------
// host
// ----------------------------------------------------------------------------
namespace {

// Workgroups of a pass over the whole call: 6 of 4 waves per compute unit. A static share wants all of them
// resident (2048 of them ran 4-6% longer than 1536), and most passes' registers allow 6 or more. The sums of fp32
// are the exception: 7, 8 and more ranks allow 5 workgroups on a compute unit, with the buckets' own norms 4, 6
// and 7 ranks allow 5, 8 and more 4. In such a pass over a full grid the others start when those have ended.
int64_t most_blocks() { return 6 * int64_t(device_cus()); }

// Work items hold a multiple of kItemUnit elements: enough of them that a workgroup's share is many (the
// shares then end together, however the tensors' last items fall), at most kMaxItem elements apiece
// where that many items are not too many to count. The kernels count an item's elements in an int: 2^30 is the
// most (2^48 elements with their own norms, the longest call, are then 2^18 items and their tensors' ends).
constexpr int64_t kItemUnit = 2048, kMaxItem = 16384, kShare = 8, kEachItems = 16384, kMostItems = int64_t(1) << 24;
constexpr int64_t kLongestItem = int64_t(1) << 30;
constexpr int64_t kPlainBlocks = 1536;  // the items' size follows the call alone, not the device
int64_t item_size(int64_t total, bool each) {
  int64_t per = std::min(kMaxItem, total / (kPlainBlocks * kShare));
  per = std::min(kLongestItem, std::max(per, total / (each ? kEachItems : kMostItems)));
  return std::max<int64_t>(1, (per + kItemUnit - 1) / kItemUnit) * kItemUnit;
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
  if (st == hipStreamPerThread) {  // one handle for every thread's stream
    r.status = 2;
    r.message = "a call on hipStreamPerThread needs a workspace of its own (" + std::to_string(need) + " bytes)";
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

// Workgroups of a launch. Their counts of items may differ by one: as many workgroups on every compute
// unit matter more (7 x 2^24 fp32: 175 us with 1536 workgroups of 5 or 6 items, 184 with 1366 of 6).
int64_t blocks_for(int64_t items) { return std::max<int64_t>(1, std::min({items, most_blocks(), launch_blocks()})); }

// Where a call's partials lie behind kHead: one per workgroup of its launches, then (each) one per wave and
// item. The size is that of launches with all of their workgroups.
struct Partials {
  std::vector<int64_t> blocks;  // workgroups of every launch
  int32_t count = 0;            // partials of workgroups
};
size_t partial_bytes(int64_t items, int64_t launches, bool each) {
  return round_up(size_t(std::min(items, launches * most_blocks()) + (each ? items * kWaves : 0)) * sizeof(double));
}
template <typename TAB> Partials place_partials(std::vector<TAB>& tabs) {
  Partials r;
  for (TAB& t : tabs) {
    r.blocks.push_back(blocks_for(t.first[t.count]));
    t.at = r.count;
    r.count += int32_t(r.blocks.back());
  }
  return r;
}
// Whether a pass that scales is to join this many partials in every workgroup: two launches' worth of them.
bool few_partials(int64_t count) { return count <= 2 * most_blocks(); }

#define AR_KIND(kind, ...)                                   \
  if ((kind) == N_L2) { constexpr int KIND = N_L2; __VA_ARGS__; } \
  else { constexpr int KIND = N_MAX; __VA_ARGS__; }

// The norm of the call, and every tensor's or bucket's own before it (clip.each; firsts: their first items).
int64_t final_cap() { return std::min<int64_t>(kEachTensors, launch_blocks()); }
int64_t final_launches(const Clip& clip, int64_t count, int64_t cap) { return pieces((clip.each ? count : 0) + 1, cap); }
void launch_final(Sequence& s, const Clip& clip, const std::vector<int32_t>& firsts, int64_t cap, const double* partial, int partials, const double* own, double* joined) {
  const int64_t count = clip.each ? int64_t(firsts.size()) - 1 : 0;
  for (int64_t i0 = 0; i0 <= count; i0 += cap) {
    EachTab tab;
    const int64_t blocks = std::min(cap, count + 1 - i0);
    tab.count = int32_t(std::min(cap, count - i0));
    for (int k = 0; k <= tab.count; ++k) tab.first[k] = firsts[size_t(i0 + k)] * kWaves;
    AR_KIND(clip.norm, s.launch(k_norm_final<KIND>, blocks, kFinalThreads, tab, partial, partials, own, joined, clip.total, clip.each + i0));
  }
}

int64_t total_of(const Grad* g, int64_t count) {
  int64_t t = 0;
  for (int64_t i = 0; i < count; ++i) t += g[i].n;
  return t;
}

// Whether one workgroup takes the whole list: one launch and no workspace, about 2 us of the host's time,
// against two launches, whose many waves soon make up for the second. Norm, fp32: 24 items 4.7 us on the
// GPU (two launches 5.5), 48 items 6.4 (5.5); with the scaling 12 items 6.3 (6.5), 24 items 8.5 (6.6).
bool small_list(int64_t count, int64_t items, bool scale) { return count <= kTabTensors && items <= (scale ? kSmallWaves : kSmallItems); }

}  // namespace

size_t grad_workspace(const Grad* g, int64_t count, const Clip& clip) {
  if (clip.known) return 0;
  const int64_t per = item_size(total_of(g, count), clip.each);
  int64_t items = 0;
  for (int64_t i = 0; i < count; ++i) items += pieces(g[i].n, per);
  if (small_list(count, items, true)) return 0;  // enough for either call
  return kHead + partial_bytes(items, pieces(count, kTabTensors), clip.each);
}

RunResult run_grad(const Grad* g, int64_t count, const Clip& clip, bool scale, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t per = item_size(total_of(g, count), clip.each);
  std::vector<GradTab> tabs;
  std::vector<int32_t> firsts{0};
  for (int64_t i0 = 0; i0 < count; i0 += kTabTensors) {
    GradTab tab;
    std::memset(&tab, 0, sizeof(tab));
    tab.count = int32_t(std::min<int64_t>(kTabTensors, count - i0));
    tab.item0 = firsts.back();
    tab.per = per;
    for (int k = 0; k < tab.count; ++k) {
      const Grad& t = g[i0 + k];
      tab.src[k] = t.data;
      tab.dst[k] = t.out;
      tab.n4[k] = (t.n << 2) | (t.out_dtype == D_BF16 ? 2 : 0) | (t.dtype == D_BF16 ? 1 : 0);
      tab.first[k + 1] = tab.first[k] + int32_t(pieces(t.n, per));
      firsts.push_back(tab.item0 + tab.first[k + 1]);
    }
    if (tab.first[tab.count] || count <= kTabTensors) tabs.push_back(tab);
  }
  const int32_t items = firsts.back();
  Sequence s{st, {reinterpret_cast<hipEvent_t>(clip.start_event), reinterpret_cast<hipEvent_t>(clip.stop_event)}, 0};
  if (!clip.known && small_list(count, items, scale)) {
    GradTab none;
    none.count = 0;
    none.first[0] = 0;
    const GradTab& t = tabs.empty() ? none : tabs[0];
    s.left = 1;
    if (scale) { AR_KIND(clip.norm, s.launch(k_grad_small<KIND, true>, 1, kSmallThreads, t, clip.total, clip.each, clip.max_norm, clip.eps)); }
    else { AR_KIND(clip.norm, s.launch(k_grad_small<KIND, false>, 1, kSmallThreads, t, clip.total, clip.each, clip.max_norm, clip.eps)); }
    return s.done("launching the gradient kernels");
  }
  const Partials parts = place_partials(tabs);
  std::unique_lock<std::mutex> lk;
  char* ws = nullptr;
  if (!clip.known) {
    const RunResult r = workspace_of(clip, grad_workspace(g, count, clip), st, lk, &ws);
    if (r.status) return r;
  }
  double* joined = reinterpret_cast<double*>(ws);  // (none of them with a known norm)
  double* partial = ws ? reinterpret_cast<double*>(ws + kHead) : nullptr;
  double* own = ws ? partial + parts.count : nullptr;
  const int64_t nt = int64_t(tabs.size());
  const bool final = !clip.known && (!scale || clip.each || !nt || !few_partials(parts.count));  // otherwise the scaling pass joins them
  const int64_t cap = final_cap();
  s.left = (clip.known ? 0 : nt) + (scale ? nt : 0) + (final ? final_launches(clip, count, cap) : 0);
  if (!clip.known)
    for (int64_t k = 0; k < nt; ++k) {
      if (clip.each) { AR_KIND(clip.norm, s.launch(k_grad_norm<KIND, true, true>, parts.blocks[k], kThreads, tabs[k], partial, own)); }
      else if (!scale) { AR_KIND(clip.norm, s.launch(k_grad_norm<KIND, false, true>, parts.blocks[k], kThreads, tabs[k], partial, own)); }
      else { AR_KIND(clip.norm, s.launch(k_grad_norm<KIND, false, false>, parts.blocks[k], kThreads, tabs[k], partial, own)); }
    }
  if (final) launch_final(s, clip, firsts, cap, partial, parts.count, own, joined);
  if (scale) {
    Limit lim{final ? joined : partial, final ? 1 : parts.count, clip.max_norm, clip.eps, clip.known, final ? nullptr : clip.total,
              std::all_of(g, g + count, [](const Grad& t) { return t.out == t.data; })};
    for (int64_t k = nt - 1; k >= 0; --k) {
      AR_KIND(clip.norm, s.launch(k_grad_scale<KIND>, parts.blocks[k], kThreads, tabs[k], lim));
      lim.total = nullptr;
    }
  }
  return s.done("launching the gradient kernels");
}

namespace {

// Few elements are cut finer and, of many ranks, 16 loaded together: what such a call waits for is one
// batch of loads after the other. us for a call in a graph, without and with that: 127 ranks x 2250 fp32
// 29.3 and 22.8, 24 x 60000 11.5 and 10.3, 192 x 65536 bf16 40.9 and 28.0, 64 x 2^18 22.2 and 19.3, 8 x 65536
// fp32 8.3 and 7.8; past the limit 8 x 2^19 fp32 12.5 and 13.1, 192 x 2^20 bf16 154 and 156.
constexpr int64_t kFineUnit = 512, kFineTotal = int64_t(1) << 18;

// Ranks that the second pass reads again rather than finding their sums (30 M elements a rank, kept
// and read again, us a call in a graph): fp32 2 ranks 128 and 125, 3 ranks 168 and 187; bf16 2 ranks 87 and 68,
// 3 ranks 111 and 97, 4 ranks 131 and 127. The reduce-scatter: fp32 2 ranks 111 and 108, 3 ranks 135 and 150;
// bf16 3 ranks 86 and 77, 4 ranks 101 and 99.
constexpr int32_t most_reread(int dtype) { return dtype == D_BF16 ? 3 : 2; }

template <int DT, int KIND, bool EACH> void launch_reduce(Sequence& s, int64_t blocks, const BucketTab& t, double* partial, double* own) {
#define AR_REDUCE_B(B_) s.launch(k_bucket_reduce<DT, KIND, B_, kPair<DT>, EACH, true>, blocks, kThreads, t, partial, own)
  if (t.P <= most_reread(DT)) {
    switch (t.P) {
      case 1: s.launch(k_bucket_reduce<DT, KIND, 1, kPair<DT>, EACH, false>, blocks, kThreads, t, partial, own); break;
      case 2: s.launch(k_bucket_reduce<DT, KIND, 2, kPair<DT>, EACH, false>, blocks, kThreads, t, partial, own); break;
      default: if constexpr (DT == D_BF16) s.launch(k_bucket_reduce<DT, KIND, 3, kPair<DT>, EACH, false>, blocks, kThreads, t, partial, own);
    }
    return;
  }
  switch (t.P <= 8 ? t.P : t.per == kFineUnit ? 16 : 8) {
    case 3: if constexpr (DT == D_FP32) AR_REDUCE_B(3); break;
    case 4: AR_REDUCE_B(4); break;
    case 5: AR_REDUCE_B(5); break;
    case 6: AR_REDUCE_B(6); break;
    case 7: AR_REDUCE_B(7); break;
    case 16: s.launch(k_bucket_reduce<DT, KIND, 16, 1, EACH, true>, blocks, kThreads, t, partial, own); break;
    default: AR_REDUCE_B(8); break;
  }
#undef AR_REDUCE_B
}

template <int DT, int KIND> void launch_spread(Sequence& s, int64_t blocks, const BucketTab& t, const Limit& lim) {
  if (t.P > most_reread(DT)) {
    s.launch(k_bucket_spread<DT, KIND, 0>, blocks, kThreads, t, lim);
    return;
  }
  switch (t.P) {
    case 1: s.launch(k_bucket_spread<DT, KIND, 1>, blocks, kThreads, t, lim); break;
    case 2: s.launch(k_bucket_spread<DT, KIND, 2>, blocks, kThreads, t, lim); break;
    default: if constexpr (DT == D_BF16) s.launch(k_bucket_spread<DT, KIND, 3>, blocks, kThreads, t, lim);
  }
}

struct BucketPlan {
  std::vector<BucketTab> tabs;
  std::vector<int32_t> firsts{0};
  int64_t launches = 0;
  size_t low_bytes = 0;  // lower halves kept in the workspace
};

bool low_in_workspace(const Buckets& b) { return b.dtype == D_BF16 && b.coll == C_REDUCE_SCATTER && b.P > most_reread(b.dtype); }

int rank_stride(int P) { return (P + kRankBatch - 1) / kRankBatch * kRankBatch; }

BucketPlan plan_buckets(const Buckets& b, int64_t per) {
  BucketPlan pl;
  const int stride = rank_stride(b.P);
  const int64_t fit = std::min<int64_t>(kTabBuckets, kTabPtrs / stride);
  const bool scatter = b.coll == C_REDUCE_SCATTER;
  for (int64_t i0 = 0; i0 < b.count; i0 += fit) {
    BucketTab tab;
    std::memset(&tab, 0, sizeof(tab));
    tab.count = int32_t(std::min(fit, b.count - i0));
    tab.P = b.P;
    tab.stride = stride;
    tab.item0 = pl.firsts.back();
    tab.owners = scatter;
    tab.per = per;
    tab.div = b.op == O_AVG ? float(b.P) : 0.0f;
    for (int k = 0; k < tab.count; ++k) {
      const int64_t n = b.n[i0 + k], part = scatter ? pieces(n, b.P) : n;
      for (int q = 0; b.bufs && q < stride; ++q) tab.p[k * stride + q] = b.bufs[(i0 + k) * b.P + std::min(q, b.P - 1)];  // none: only the size is asked
      tab.n[k] = n;
      tab.part[k] = part;
      tab.ipp[k] = int32_t(std::max<int64_t>(1, pieces(part, per)));
      if (low_in_workspace(b)) {
        tab.low[k] = reinterpret_cast<uint16_t*>(pl.low_bytes);  // an offset until the workspace is known
        pl.low_bytes += round_up(size_t(n) * 2);
      } else if (b.dtype == D_BF16 && b.P > most_reread(b.dtype)) {
        tab.low[k] = static_cast<uint16_t*>(tab.p[k * stride + 1]);
      }
      tab.first[k + 1] = tab.first[k] + (n ? tab.ipp[k] * (scatter ? b.P : 1) : 0);
      pl.firsts.push_back(tab.item0 + tab.first[k + 1]);
    }
    if (tab.first[tab.count] || b.count <= fit) pl.tabs.push_back(tab);
  }
  pl.launches = int64_t(pl.tabs.size());
  return pl;
}

// The call's plan; small: one workgroup takes all of it.
BucketPlan plan_call(const Buckets& b, bool each, bool* small) {
  const bool scatter = b.coll == C_REDUCE_SCATTER;
  int64_t total = 0, items = 0;
  for (int64_t i = 0; i < b.count; ++i) {
    total += b.n[i];
    if (b.n[i]) items += scatter ? b.P * pieces(pieces(b.n[i], b.P), kSmallSpan) : pieces(b.n[i], kSmallSpan);
  }
  *small = b.count <= std::min<int64_t>(kTabBuckets, kTabPtrs / rank_stride(b.P)) && items <= kSmallWaves;
  return plan_buckets(b, *small ? kSmallSpan : total <= kFineTotal ? kFineUnit : item_size(total, each));
}

// Where the lower halves start, behind the partials.
size_t low_offset(const BucketPlan& pl, bool each) { return kHead + partial_bytes(pl.firsts.back(), pl.launches, each); }

}  // namespace

size_t allreduce_clip_workspace(const Buckets& b, const Clip& clip) {
  bool small;
  const BucketPlan pl = plan_call(b, clip.each, &small);
  return small ? 0 : low_offset(pl, clip.each) + pl.low_bytes;
}

RunResult run_allreduce_clip(const Buckets& b, const Clip& clip, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  bool small;
  BucketPlan pl = plan_call(b, clip.each, &small);
  Sequence s{st, {reinterpret_cast<hipEvent_t>(clip.start_event), reinterpret_cast<hipEvent_t>(clip.stop_event)}, 0};
  if (small) {
    BucketTab none;
    std::memset(&none, 0, sizeof(none));
    const BucketTab& t = pl.tabs.empty() ? none : pl.tabs[0];
    s.left = 1;
    if (b.dtype == D_BF16) { AR_KIND(clip.norm, s.launch(k_bucket_small<D_BF16, KIND>, 1, kSmallThreads, t, clip.total, clip.each, clip.max_norm, clip.eps)); }
    else { AR_KIND(clip.norm, s.launch(k_bucket_small<D_FP32, KIND>, 1, kSmallThreads, t, clip.total, clip.each, clip.max_norm, clip.eps)); }
    return s.done("launching the gradient kernels");
  }
  std::unique_lock<std::mutex> lk;
  char* ws = nullptr;
  const RunResult r = workspace_of(clip, low_offset(pl, clip.each) + pl.low_bytes, st, lk, &ws);
  if (r.status) return r;
  double* joined = reinterpret_cast<double*>(ws);
  double* partial = reinterpret_cast<double*>(ws + kHead);
  const Partials parts = place_partials(pl.tabs);
  double* own = partial + parts.count;
  char* low = ws + low_offset(pl, clip.each);
  for (BucketTab& t : pl.tabs)
    for (int k = 0; low_in_workspace(b) && k < t.count; ++k)
      t.low[k] = reinterpret_cast<uint16_t*>(low + reinterpret_cast<size_t>(t.low[k]));
  const int64_t nt = int64_t(pl.tabs.size());
  const bool final = clip.each || !nt || !few_partials(parts.count);  // otherwise the second pass joins them
  const int64_t cap = final_cap();
  s.left = 2 * nt + (final ? final_launches(clip, b.count, cap) : 0);
  for (int64_t k = 0; k < nt; ++k) {
#define AR_REDUCE(DT_, EACH_) AR_KIND(clip.norm, launch_reduce<DT_, KIND, EACH_>(s, parts.blocks[k], pl.tabs[k], partial, own))
    if (b.dtype == D_BF16) {
      if (clip.each) { AR_REDUCE(D_BF16, true); } else { AR_REDUCE(D_BF16, false); }
    } else {
      if (clip.each) { AR_REDUCE(D_FP32, true); } else { AR_REDUCE(D_FP32, false); }
    }
#undef AR_REDUCE
  }
  if (final) launch_final(s, clip, pl.firsts, cap, partial, parts.count, own, joined);
  Limit lim{final ? joined : partial, final ? 1 : parts.count, clip.max_norm, clip.eps, nullptr, final ? nullptr : clip.total, false};
  for (int64_t k = 0; k < nt; ++k) {
    if (b.dtype == D_BF16) { AR_KIND(clip.norm, launch_spread<D_BF16, KIND>(s, parts.blocks[k], pl.tabs[k], lim)); }
    else { AR_KIND(clip.norm, launch_spread<D_FP32, KIND>(s, parts.blocks[k], pl.tabs[k], lim)); }
    lim.total = nullptr;
  }
  return s.done("launching the gradient kernels");
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

RunResult grad_cache_wait() {
  std::lock_guard<std::mutex> lk(g_mu);
  std::set<int> devices;
  for (const auto& kv : kept()) devices.insert(kv.first.first);
  for (const Kept& w : retired()) devices.insert(w.device);
  if (devices.empty()) return RunResult{};
  int current = 0;
  hipError_t e = hipGetDevice(&current);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  for (int d : devices) {
    e = hipSetDevice(d);
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) break;
  }
  (void)hipSetDevice(current);
  return e == hipSuccess ? RunResult{} : hip_fail(e, "synchronizing before the release");
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
