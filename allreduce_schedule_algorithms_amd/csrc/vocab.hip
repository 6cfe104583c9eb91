// Losses over a vocabulary in pieces for gfx950: softmax cross entropy and the distance
// to a teacher's top logits, of hidden states h [T, H] against an output matrix W [V, H]
// whose rows lie in P pieces, and their gradients.
//
//   z = h W^T / temperature                       (not kept; with gradients its exponentials are, a chunk of tokens' at a time)
//   lse_t = log(sum_v exp z_tv),  p = exp(z - lse)
//   cross entropy:  loss_t = lse_t - z_ty
//   distillation:   q_t = softmax(teacher / temperature),
//                   loss_t = sum_k q_tk (log q_tk - z_t,id(k) + lse_t)
//   D = c (p - q)   with q the one-hot target for cross entropy, c_t the row's weight in
//                   the call's loss over the temperature
//   dh = D W,  dW = D^T h
//
// (In bf16 D is rounded, of few rows to two bf16 terms. 1 / N of a mean over N rows, the same in every D, would be rounded the same way in all of
// them, which no sum over rows or ids evens out: of c, D takes on a power of two, and the results the rest.)
//
// Rows that the targets leave out take no part: the rows that count are gathered in order
// (k_vocab_prepare, k_vocab_pack), and every product runs over as many as there are. The products are
// matrix products of bf16 operands with fp32 sums; fp32 operands are split exactly into
// three bf16 terms each, and the six products of the larger terms are summed (what is
// left out is 2^-26 of a product).
//
// A call works on the tokens in chunks, so that its scratch is bounded: the logits' tile
// leaves the product as exp(z - m), m the row's largest of the tile, beside m and the tile's sum; once
// a row's lse is known, one pass turns them into D. Nothing is added atomically: the
// same sizes give the same bits on every run.
//
// 8192 tokens x 4096 x 128000 in bf16, 8 pieces, with gradients: 21.1 ms, of which products 6.88 + 6.51 + 6.91
// (1249, 1321 and 1244 TFLOP/s), D 0.74, the rest 0.07. (Cards differ by some 3%.)
#include "vocab.h"

#include <hip/hip_ext.h>

#include <algorithm>

#include "kernels.h"
#include "sequence.h"

namespace ar {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
#define AR_LDS __attribute__((address_space(3)))

constexpr int kBK = 32;         // depth of a slice: one product's, 64 bytes of a row
constexpr int kPieceTab = 64;   // pieces that one launch's arguments carry
constexpr int kUnit = 256;      // pieces and token chunks are padded to this many rows
constexpr float kLn2 = 0.69314718055994530942f;  // logs are in units of it

// One piece as the kernels see it, in the workspace. `first`: its first row in the vocabulary; `start`: the same
// with every piece padded to kUnit rows, the coordinate that tiles, D and the ids' table use.
struct Piece {
  const char* w;
  char* dw;
  int64_t ld, dld;
  int32_t rows, start, first, pad;
};

struct PieceTab {
  Piece p[kPieceTab];
  int32_t count, at;
};

struct alignas(16) Counts {
  int32_t active;  // rows that take part
  int32_t mean;    // rows that are not left out (those of weight 0 among them)
  int32_t bad;     // rows with an id outside the vocabulary
  float factor;    // what a mean and the temperature make of the gradients is share times factor: a power of two, which D
  double share;    // takes on, and a value in [1, 2), which the results are multiplied by in fp32
};

enum Flag : uint8_t { F_OUT = 0, F_ACTIVE = 1, F_BAD = 2, F_ZERO = 3 };

template <bool BY_START> __device__ __forceinline__ int piece_of(const Piece* p, int P, int32_t at) {
  int lo = 0, hi = P;  // the last piece that begins at or before `at`
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if ((BY_START ? p[mid].start : p[mid].first) <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int64_t id_at(const void* ids, bool wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(ids)[i] : int64_t(static_cast<const int32_t*>(ids)[i]);
}

__device__ __forceinline__ float logit_at(const void* p, int dtype, int64_t i) {
  return dtype == D_BF16 ? as_f(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16) : static_cast<const float*>(p)[i];
}

// x as a sum of three bf16 values, exactly: each is the nearest to what is left (a magnitude that would round to
// an infinity is cut instead), and 24 bits leave at most 8 for the third.
__device__ __forceinline__ void split3(float x, __bf16 (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    __bf16 b = __bf16(x);
    if (__builtin_isinf(float(b)) && !__builtin_isinf(x)) b = __builtin_bit_cast(__bf16, uint16_t(as_u(x) >> 16));
    t[i] = b;
    x = __builtin_isfinite(float(b)) ? x - float(b) : 0.f;  // infinities and NaN stay in the first term
  }
}

// The same of N values, two at a time: the rare magnitudes that round to an infinity, infinities and NaN take the
// way above.
template <int N, class V, class B> __device__ __forceinline__ void split3_of(const V& x, B (&t)[3]) {
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) most = max(most, as_u(x[j]) & 0x7fffffffu);
  if (most < 0x7f7f8000u) {
    V r = x;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      t[i] = __builtin_convertvector(r, B);
      r -= __builtin_convertvector(t[i], V);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      __bf16 b[3];
      split3(x[j], b);
#pragma unroll
      for (int i = 0; i < 3; ++i) t[i][j] = b[i];
    }
  }
}

// ----------------------------------------------------------------------------
// rows
// ----------------------------------------------------------------------------
// What a call's targets are.
struct Targets {
  const void* ids;
  const void* logits;
  const float* weights;
  int64_t ids_ld, logits_ld, ignore, V;
  int32_t K, logits_dtype;  // K = 0: one target a row
  bool wide;
  float temperature;
};

// Distillation: a wave per row finds the teacher's largest logit and the sum of exp around it. Logits are divided by the
// temperature as differences to the largest: their own quotients may pass the largest fp32 value.
constexpr int kRowWaves = 4;
__global__ __launch_bounds__(kRowWaves * 64) void k_vocab_teacher(Targets t, int64_t T, float2* stat, uint8_t* flags) {
  const int lane = threadIdx.x & 63;
  for (int64_t r = int64_t(blockIdx.x) * kRowWaves + threadIdx.x / 64; r < T; r += int64_t(gridDim.x) * kRowWaves) {
    float top = -INFINITY;
    bool bad = false, nan = false;
    for (int k = lane; k < t.K; k += 64) {
      const int64_t id = id_at(t.ids, t.wide, r * t.ids_ld + k);
      if (id < 0) continue;
      bad |= id >= t.V;
      const float x = logit_at(t.logits, t.logits_dtype, r * t.logits_ld + k);
      nan |= x != x;
      top = fmaxf(top, x);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    bad = __any(bad);
    nan = __any(nan);
    if (nan) top = NAN;
    float sum = 0;
    for (int k = lane; k < t.K; k += 64)
      if (id_at(t.ids, t.wide, r * t.ids_ld + k) >= 0)
        sum += expf((logit_at(t.logits, t.logits_dtype, r * t.logits_ld + k) - top) / t.temperature);
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) {
      stat[r] = float2{top, sum};
      // no entries, or none above -infinity: the row has no distribution and is left out
      flags[r] = bad ? F_BAD : top == -INFINITY ? F_OUT : t.weights && t.weights[r] == 0 ? F_ZERO : F_ACTIVE;
    }
  }
}

// Rows that take part, in order, at rows[0..active); the others behind them. One workgroup; returns active.
constexpr int kScanThreads = 1024, kScanEach = 4;
__device__ __forceinline__ int scan_rows(const Targets& t, int64_t T, bool mean_of, int32_t* rows, uint8_t* flags, Counts* counts) {
  __shared__ int wave_n[kScanThreads / 64][kScanEach], tally[2], round;
  const int tid = threadIdx.x, wave = tid / 64, lane = tid & 63;
  if (tid < 2) tally[tid] = 0;
  int done = 0, mean = 0, bad = 0;  // active rows before this round; the thread's own tallies
  for (int64_t base = 0; base < T; base += kScanThreads * kScanEach) {
    uint8_t f[kScanEach];
    uint64_t mask[kScanEach];
#pragma unroll
    for (int j = 0; j < kScanEach; ++j) {
      const int64_t r = base + j * kScanThreads + tid;
      f[j] = F_OUT;
      if (r < T) {
        if (t.K) {
          f[j] = flags[r];
        } else {
          const int64_t id = id_at(t.ids, t.wide, r);
          f[j] = id == t.ignore ? F_OUT : id < 0 || id >= t.V ? F_BAD : t.weights && t.weights[r] == 0 ? F_ZERO : F_ACTIVE;
          flags[r] = f[j];
        }
        mean += f[j] != F_OUT;
        bad += f[j] == F_BAD;
      }
      mask[j] = __ballot(f[j] == F_ACTIVE);
      if (lane == 0) wave_n[wave][j] = __popcll(mask[j]);
    }
    __syncthreads();
    if (wave == 0) {  // a lane for every wave and round, in the rows' order: what comes before it
      static_assert(kScanThreads / 64 * kScanEach == 64, "one wave adds all counts up");
      const int w = lane % (kScanThreads / 64), j = lane / (kScanThreads / 64), n = wave_n[w][j];
      int upto = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d);
        upto += lane >= d ? o : 0;
      }
      wave_n[w][j] = upto - n;
      if (lane == 63) round = upto;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kScanEach; ++j) {
      const int64_t r = base + j * kScanThreads + tid;
      const int mine = done + wave_n[wave][j] + __popcll(mask[j] & ((uint64_t(1) << lane) - 1));  // active rows before r
      if (r < T) {
        if (f[j] == F_ACTIVE) rows[mine] = int32_t(r);
        else rows[T - 1 - (r - mine)] = int32_t(r);  // r - mine others before it: from the end
      }
    }
    done += round;
    __syncthreads();
  }
  if (mean) atomicAdd(&tally[0], mean);  // whole numbers in LDS: the order does not matter
  if (bad) atomicAdd(&tally[1], bad);
  __syncthreads();
  if (tid == 0) {
    int e;
    const double m = frexp(1 / (double(t.temperature) * (mean_of && tally[0] ? tally[0] : 1)), &e);
    *counts = Counts{done, tally[0], tally[1], float(2 * m), ldexp(1., e - 1)};
  }
  __syncthreads();
  return done;
}

// The hidden rows that take part, gathered as bf16 terms of Hp elements each, zeros behind them; their ids as padded
// coordinates; and what the rows left out get: gradients and losses of 0 (NaN where an id is outside).
struct PackArgs {
  const void* hidden;
  int64_t ld, T, Tpad;
  int32_t H, Hp, P;
  const Piece* pieces;
  const int32_t* rows;
  const uint8_t* flags;
  const Counts* counts;
  char* hp;
  int32_t* idt;  // [Tpad][Kp], -1 behind a row's ids
  int32_t Kp;
  int32_t lo;    // as in Product: the rows are there once more from this one on
  void* dh;      // null: no gradient
  int64_t dh_ld;
  float* each;   // every row's loss, or null
};

// A row of H elements into terms of Hp elements, zero behind H. Called by a whole wave; four vectors a lane are on
// their way together.
template <int DT> __device__ __forceinline__ void pack_row(const void* src, int64_t at, int H, int Hp, __bf16* dst, int lane) {
  using E = std::conditional_t<DT == D_BF16, uint16_t, float>;
  typedef E V __attribute__((ext_vector_type(8)));
  typedef E Any __attribute__((ext_vector_type(8), aligned(sizeof(E))));
  const E* s = static_cast<const E*>(src) + at;
  for (int c0 = lane * 8; c0 < Hp; c0 += 4 * 512) {
    V v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = c0 + q * 512;
      v[q] = V{};
      if (c + 8 <= H) {
        v[q] = *reinterpret_cast<const Any*>(s + c);
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (c + j < H) v[q][j] = s[c + j];
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = c0 + q * 512;
      if (c >= Hp) break;
      if constexpr (DT == D_BF16) {
        *reinterpret_cast<V*>(dst + c) = v[q];
      } else {
        bf16x8 o[3];
        split3_of<8>(v[q], o);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x8*>(dst + int64_t(i) * Hp + c) = o[i];
      }
    }
  }
}

template <int DT> __device__ __forceinline__ void pack_rows(const PackArgs& a, const Targets& t, const Piece* pieces, int active, int64_t first, int64_t step) {
  constexpr int PL = DT == D_FP32 ? 3 : 1;
  const int lane = threadIdx.x & 63;
  // the products go 2 kBK rows deep at a time, and tiles look up the ids of up to kUnit rows
  const int lo = DT == D_BF16 ? a.lo : 0, zeros = lo ? 2 * lo : (active + 2 * kBK - 1) / (2 * kBK) * 2 * kBK, end = (active + kUnit - 1) / kUnit * kUnit;
  const int K = t.K ? t.K : 1;
  for (int64_t i = first; i < a.Tpad; i += step) {
    const int64_t r = i < a.T ? a.rows[i] : -1;
    __bf16* dst = reinterpret_cast<__bf16*>(a.hp) + i * PL * a.Hp;
    int64_t from = i < active ? r : -1;
    if (lo && i >= lo && i < lo + active) from = a.rows[i - lo];
    if (from >= 0) {
      pack_row<DT>(a.hidden, from * a.ld, a.H, a.Hp, dst, lane);
    } else if (i < zeros) {
      for (int c = lane * 8; c < PL * a.Hp; c += 512) *reinterpret_cast<bf16x8*>(dst + c) = bf16x8{};
    }
    if (i < end)
      for (int k = lane; k < a.Kp; k += 64) {
        int32_t at = -1;
        if (i < active && k < K) {
          const int64_t id = t.K ? id_at(t.ids, t.wide, r * t.ids_ld + k) : id_at(t.ids, t.wide, r);
          if (id >= 0) {
            const Piece& p = pieces[piece_of<false>(pieces, a.P, int32_t(id))];
            at = p.start + int32_t(id) - p.first;
          }
        }
        a.idt[i * a.Kp + k] = at;
      }
    if (i >= active && r >= 0) {
      if (a.each && lane == 0) a.each[r] = a.flags[r] == F_BAD ? NAN : 0.f;
      if (a.dh)
        for (int c = lane; c < a.H; c += 64) {
          if constexpr (DT == D_BF16) static_cast<uint16_t*>(a.dh)[r * a.dh_ld + c] = 0;
          else static_cast<float*>(a.dh)[r * a.dh_ld + c] = 0;
        }
    }
  }
}
template <int DT> __global__ __launch_bounds__(kRowWaves * 64) void k_vocab_pack(PackArgs a, Targets t) {
  pack_rows<DT>(a, t, a.pieces, a.counts->active, int64_t(blockIdx.x) * kRowWaves + threadIdx.x / 64, int64_t(gridDim.x) * kRowWaves);
}

// More ids a row than kFewIds are sorted by the tile of logits that they lie in, so that a tile finds its own: one
// workgroup for the rows of a tile counts them, adds the counts up and deals the entries out. (Where an entry lies
// among its tile's does not show in any result.) 3687 rows x 64 ids: 22 us, after which the logits of 50000 took 886;
// with tiles that compare all of their rows' ids, 1176.
constexpr int kFewIds = 4, kSortThreads = 1024;
__global__ __launch_bounds__(kSortThreads) void k_vocab_sort(const int32_t* idt, int ld_idt, int bn, int bm, int mtiles, int64_t row_tiles, const Counts* counts, int32_t* starts, uint32_t* entries) {
  extern __shared__ int32_t place[];  // [mtiles + 1]
  __shared__ int32_t wave_sum[kSortThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  for (int64_t t = blockIdx.x; t < row_tiles && t * bn < counts->active; t += gridDim.x) {
    for (int i = tid; i <= mtiles; i += kSortThreads) place[i] = 0;
    __syncthreads();
    const int32_t* ids = idt + t * bn * ld_idt;
    const int all = bn * ld_idt;
    for (int i = tid; i < all; i += kSortThreads)
      if (ids[i] >= 0) atomicAdd(&place[ids[i] / bm], 1);
    __syncthreads();
    const int per = (mtiles + 1 + kSortThreads - 1) / kSortThreads, i0 = min(tid * per, mtiles + 1), i1 = min(i0 + per, mtiles + 1);
    int mine = 0;
    for (int i = i0; i < i1; ++i) mine += place[i];
    int before = mine;  // this thread's and the earlier ones' of the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(before, d);
      before += lane >= d ? o : 0;
    }
    if (lane == 63) wave_sum[tid / 64] = before;
    __syncthreads();
    int at = before - mine;
    for (int w = 0; w < tid / 64; ++w) at += wave_sum[w];
    for (int i = i0; i < i1; ++i) {
      const int n = place[i];
      place[i] = at;
      starts[t * (mtiles + 1) + i] = at;
      at += n;
    }
    __syncthreads();
    for (int i = tid; i < all; i += kSortThreads) {
      const int32_t id = ids[i];
      if (id >= 0) entries[t * all + atomicAdd(&place[id / bm], 1)] = uint32_t(id % bm) | uint32_t(i / ld_idt) << 8 | uint32_t(i % ld_idt) << 16;
    }
    __syncthreads();
  }
}

// A call's first launch (one for every kPieceTab pieces). Workgroup 0 writes the products' table of pieces and finds
// the rows that take part (and packs them: few elements, which another launch would cost more than). The others copy
// the output matrix as bf16 terms where the products cannot read it (fp32, and bf16 that 16-byte loads do not fit):
// row v of the padded vocabulary at wp + v * PL * Hp. Bound by memory: 131 MB of fp32 into 197 MB take 58 us, 5.6 TB/s.
struct PrepareArgs {
  PieceTab tab;
  Piece* pieces;
  char* wp;  // null: read in place
  int32_t scan, pack, mean, H, Hp;
  int64_t T;
  int32_t* rows;
  uint8_t* flags;
  Counts* counts;
};
template <int DT> __global__ __launch_bounds__(kScanThreads) void k_vocab_prepare(PrepareArgs p, Targets t, PackArgs a) {
  constexpr int PL = DT == D_FP32 ? 3 : 1;
  const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
  const int64_t row = int64_t(PL) * p.Hp;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.tab.count; i += kScanThreads) {
      Piece q = p.tab.p[i];
      if (p.wp) {
        q.w = p.wp + q.start * row * 2;
        q.ld = row;
      }
      p.pieces[p.tab.at + i] = q;
    }
    if (p.scan) {
      const int active = scan_rows(t, p.T, p.mean, p.rows, p.flags, p.counts);
      if (p.pack) pack_rows<DT>(a, t, p.tab.p, active, wave, kScanThreads / 64);
    }
  }
  if (!p.wp) return;
  const int64_t helpers = gridDim.x > 1 ? gridDim.x - 1 : 1, me = gridDim.x > 1 ? int64_t(blockIdx.x) - 1 : 0;
  if (me < 0) return;
  const Piece& last = p.tab.p[p.tab.count - 1];
  for (int64_t v = p.tab.p[0].start + me * (kScanThreads / 64) + wave; v < int64_t(last.start) + last.rows; v += helpers * (kScanThreads / 64)) {
    const Piece& q = p.tab.p[piece_of<true>(p.tab.p, p.tab.count, int32_t(v))];
    const int64_t r = v - q.start;
    if (r < q.rows) pack_row<DT>(q.w, r * q.ld, p.H, p.Hp, reinterpret_cast<__bf16*>(p.wp) + v * row, lane);
  }
}

// ----------------------------------------------------------------------------
// matrix products
// ----------------------------------------------------------------------------
// Out[n][m] = sum_k X[m][k] Y[n][k], m along the outputs' rows. Tiles of BM x BN outputs are kept by WM x WN waves
// in the accumulators of 16 x 16 x 32 products (a lane holds four consecutive m of one n); operands come through
// LDS in slices of kBK, loaded straight into it.
//
// A slice lies in LDS either as rows of 32 k (64 bytes; "along k") or as k rows of the tile's columns ("across").
// The loads write LDS in lane order, so the swizzle that spreads the reads over the banks is in which 16
// bytes a lane loads: along k, chunk c of row r lies at c ^ {0, 2, 3, 1}[r / 4 % 4]; across, the 32 bytes c of k row r lie at
// c ^ (r % 4 + 4 (r / 8 % 4)), and the reads transpose. The counters find no bank conflicts.
enum Dir { S_LOGITS = 0, S_HIDDEN = 1, S_WEIGHT = 2 };

template <int BM_, int BN_, int WM_, int WN_, int WAVES_, int STAGES_> struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, kThreads = WM * WN * 64;
  static constexpr int MW = BM / WM, NW = BN / WN;  // a wave's part
  static_assert(NW <= 64, "a lane looks after one of a wave's n");
  static constexpr int FM = MW / 16, FN = NW / 16;
  static constexpr int kWaves = WAVES_;  // of a SIMD, which bounds the registers
  static constexpr int kStages = STAGES_;  // slices in LDS, an odd number
  static constexpr int kX = BM * kBK * 2, kY = BN * kBK * 2, kStage = kX + kY;
};
using TileL = Tile<256, 256, 2, 4, 2, 5>;
using TileM = Tile<128, 128, 2, 2, 2, 5>;
using TileS = Tile<128, 64, 4, 1, 2, 5>;
// Few rows of an output matrix that is split on the way: fp32 takes three times the LDS, and half the tile.
template <int DT> using TileF = std::conditional_t<DT == D_FP32, Tile<64, 64, 4, 1, 2, 5>, TileS>;

struct Product {
  const Piece* pieces;  // the call's Counts lie before them: one address, for registers are short where this is used
  int32_t P, H, Hp, Vp, mtiles, planes;
  int32_t splits, bn, resident;  // at most so many shares of the depth; columns of a tile; workgroups that stay resident
  int32_t chunk, chunk_rows;  // this call's rows: [chunk, chunk + chunk_rows) of those that take part
  int32_t lo;                 // few rows of bf16: what D's rounding leaves, rounded too, is its rows from this one on; or 0
  int32_t kend;               // elements of a row along H that exist
  const char* hp;             // gathered hidden rows
  char* d;                    // [rows][planes * Vp]: (bf16) exp(z - m) in fp16, then D
  // logits
  float scale;  // log2(e) / temperature
  float2* stats;  // [Vp / BM][ld_stats]: a tile's largest product, the sum of 2^((product - largest) scale)
  int64_t ld_stats;
  const int32_t* idt;  // [rows][ld_idt], as zt
  int32_t ld_idt;
  float* zt;  // the products at those ids
  const int32_t* starts;    // more than kFewIds: where each tile's entries begin, [row tiles][mtiles + 1]
  const uint32_t* entries;  // [row tiles][BN ids], m | n << 8 | k << 16 within the tile
  int32_t entries_ld;
  // gradients
  const int32_t* rows;
  void* dh;
  int64_t dh_ld;
  float* part;  // fp32 partials [split][n][Hp], or null: write the outputs
  int64_t part_stride;
  int32_t accumulate;
};

typedef int32_t Rsrc __attribute__((ext_vector_type(4)));

__device__ __forceinline__ Rsrc rsrc_of(const char* base, int bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return Rsrc{int32_t(p), int32_t(p >> 32) & 0xffff, bytes, 0x00020000};
}
// s_waitcnt: all but the last n vector memory operations done, and (lds) every LDS operation.
constexpr int waits(int n, bool lds = true) { return (n & 15) | (n >> 4) << 14 | 0x70 | (lds ? 0 : 0xf00); }
constexpr int kLdsDone = 0xc07f;  // every LDS operation and scalar load done
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every buffer: such a lane loads zeros

// 16 bytes a lane straight into LDS, lane after lane. Written out because the compiler, where it knows of such a
// load, has every transposing read of LDS wait for it; here the barriers do. Nothing is written to registers.
__device__ __forceinline__ void load_lds(AR_LDS char* lds, Rsrc r, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(uint32_t(reinterpret_cast<uintptr_t>(lds))), "v"(off), "s"(r) : "memory", "m0");
}

// A read of 16 bytes a lane serves four rows of four lanes at a time, those of q = r / 4 % 4 and chunk (0, 0), (3, 0),
// (1, 1), (2, 1) or the like: with c ^ q two of them met in the same banks.
__device__ __forceinline__ uint32_t along_swizzle(uint32_t row) {
  const uint32_t q = row / 4 % 4;
  return q / 2 | ((q ^ q / 2) & 1) * 2;
}
template <int R> __device__ __forceinline__ uint32_t across_swizzle(uint32_t krow) { return (krow % 4 + krow / 8 % 4 * 4) & (R / 16 - 1); }

// How a workgroup loads a slice of R rows along k, or of R columns across: load i brings rows `kStep` further on, at
// an offset that alternates where the swizzle does.
template <int R, int THREADS, bool ALONG> struct Loads {
  static constexpr int kCount = R * kBK * 2 / (THREADS * 16), kStep = ALONG ? THREADS / 4 : THREADS / (R / 8);
  static constexpr int kOffsets = ALONG || kStep >= 32 ? 1 : 32 / kStep;
  static_assert(kStep % (ALONG ? 16 : 8) == 0 && R * kBK * 2 % (THREADS * 16) == 0, "the swizzle repeats");
  uint32_t off[kOffsets], c;

  __device__ __forceinline__ void set(uint32_t ldb, int tid) {
    if constexpr (ALONG) {
      const uint32_t row = uint32_t(tid) / 4;
      c = (uint32_t(tid) % 4) ^ along_swizzle(row);
      off[0] = row * ldb + c * 16;
    } else {
      const uint32_t krow = uint32_t(tid) / (R / 8), slot = uint32_t(tid) % (R / 8);
#pragma unroll
      for (int i = 0; i < kOffsets; ++i) off[i] = krow * ldb + (((slot / 2) ^ across_swizzle<R>(krow + i * kStep)) * 2 + slot % 2) * 16;
    }
  }
  // Of a row along k, `left` elements exist.
  __device__ __forceinline__ uint32_t at(int i, uint32_t ldb, int left) const {
    const uint32_t o = off[i % kOffsets] + i * kStep * ldb;
    return !ALONG || int(c * 8) < left ? o : kNowhere;
  }
};

// The operand of one product: 16 rows from `base`, k 8 (lane / 16) on.
__device__ __forceinline__ bf16x8 read_along(AR_LDS const char* lds, int base, int lane) {
  const int row = base + lane % 16, c = (lane / 16) ^ along_swizzle(lane);
  return *reinterpret_cast<AR_LDS const bf16x8*>(lds + row * 64 + c * 16);
}
template <int R> __device__ __forceinline__ bf16x8 read_across(AR_LDS char* lds, int base, int lane) {
  const uint32_t krow = lane / 16 * 8 + lane % 16 / 4;
  AR_LDS char* p = lds + krow * (R * 2) + ((base / 16) ^ across_swizzle<R>(krow)) * 32 + lane % 4 * 8;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((AR_LDS s16x4*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((AR_LDS s16x4*)(p + 4 * R * 2));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// Which terms of X and Y the passes over k multiply: the small ones first.
__device__ __forceinline__ int plane_x(int pass, int planes) { return planes == 1 ? 0 : (0x001102 >> (pass * 4)) & 15; }
__device__ __forceinline__ int plane_y(int pass, int planes) { return planes == 1 ? 0 : (0x010120 >> (pass * 4)) & 15; }

// A value that every lane of a wave holds, where the compiler has to know it.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(x)))) | uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(x >> 32)))) << 32);
}

// Where a product's slices come from, and the loads that bring them into LDS.
template <class C, int DIR> struct Stager {
  static constexpr bool kXAlong = DIR == S_LOGITS, kYAlong = DIR != S_WEIGHT;
  using LX = Loads<C::BM, C::kThreads, kXAlong>;
  using LY = Loads<C::BN, C::kThreads, kYAlong>;
  static constexpr int kLoads = LX::kCount + LY::kCount;
  const Product& a;
  int m0, n0, tid, steps;  // steps of one pass over the depth
  // the piece of the output matrix that is being read: its rows are [start, start + rows) of the padded vocabulary
  const char* w;
  int64_t ld;
  int rows, start, next;
  // the next slice
  int wave, pass, k, stop, slices;  // stop: the depth at which the addresses break off; slices: how many there are from it on
  const char *xp, *yp;
  int xrec;  // bytes from xp that may be read
  Rsrc x, y;
  LX lx;
  LY ly;
  uint32_t ldx, ldy;  // bytes
  int left;

  __device__ __forceinline__ void take_at(int32_t v) {
    const int p = __builtin_amdgcn_readfirstlane(piece_of<true>(a.pieces, a.P, v));
    const Piece& q = a.pieces[p];
    w = reinterpret_cast<const char*>(uniform(reinterpret_cast<int64_t>(q.w)));
    ld = uniform(q.ld);
    rows = __builtin_amdgcn_readfirstlane(q.rows);
    start = __builtin_amdgcn_readfirstlane(q.start);
    next = p + 1 < a.P ? __builtin_amdgcn_readfirstlane(a.pieces[p + 1].start) : 0x7fffffff;
    ldx = uint32_t(ld * 2);
    lx.set(ldx, tid);
  }

  __device__ __forceinline__ void begin(int m, int n) {
    m0 = m;
    n0 = n;
    start = next = 0;
    left = kBK;
    if constexpr (DIR == S_LOGITS) take_at(m0);
    if constexpr (DIR == S_WEIGHT) lx.set(ldx = uint32_t(a.planes) * uint32_t(a.Hp) * 2, tid);
    ldy = DIR == S_LOGITS ? uint32_t(a.planes) * uint32_t(a.Hp) * 2 : uint32_t(a.planes) * uint32_t(a.Vp) * 2;
    ly.set(ldy, tid);
  }

  // Points the loads at slice s of [.., end); behind the last they bring zeros.
  __device__ __forceinline__ void seek(int s, int end) {
    pass = s / steps;
    k = (s - pass * steps) * kBK;
    slices = end - s;
    find();
  }
  __device__ __forceinline__ void find() {
    const int px = plane_x(pass, a.planes), py = plane_y(pass, a.planes);
    const int64_t ldh = int64_t(a.planes) * a.Hp, ldd = int64_t(a.planes) * a.Vp;
    stop = steps * kBK;
    if constexpr (DIR == S_LOGITS) {
      const int64_t r = m0 - start;
      xp = w + (r * ld + int64_t(px) * a.Hp + k) * 2;
      left = a.kend - k;
      xrec = r < rows ? (min(rows - int(r), C::BM) - 1) * int(ldx) + left * 2 : 0;
      yp = a.hp + (int64_t(a.chunk + n0) * ldh + int64_t(py) * a.Hp + k) * 2;
    } else if constexpr (DIR == S_HIDDEN) {
      if (k < start || k >= next) take_at(k);
      stop = min(stop, next);
      xp = w + (int64_t(k - start) * ld + int64_t(px) * a.Hp + m0) * 2;
      yp = a.d + (int64_t(n0) * ldd + int64_t(py) * a.Vp + k) * 2;
    } else {
      // columns past a row's end are the next row's: they meet outputs that nothing keeps
      xp = a.hp + (int64_t(a.chunk + k) * ldh + int64_t(px) * a.Hp + m0) * 2;
      xrec = kBK * int(ldx) - (px * a.Hp + m0) * 2;
      yp = a.d + (int64_t(k) * ldd + int64_t(py) * a.Vp + n0) * 2;
    }
    describe();
  }
  __device__ __forceinline__ void describe() {
    if constexpr (DIR == S_HIDDEN) {
      const int there = min(rows - (k - start), kBK);
      xrec = there > 0 ? (there - 1) * int(ldx) + (a.kend - m0) * 2 : 0;
    }
    x = rsrc_of(xp, slices > 0 ? max(xrec, 0) : 0);  // (below 0: a tile without rows, further along its depth)
    y = rsrc_of(yp, slices > 0 ? 0x7ffffff0 : 0);
  }
  // On to the next slice; turn() has to follow wherever the addresses may break off, after every second slice (pieces
  // and passes are whole pairs of them).
  __device__ __forceinline__ void advance() {
    k += kBK;
    --slices;
    xp += DIR == S_LOGITS ? kBK * 2 : kBK * ldx;
    yp += DIR == S_WEIGHT ? kBK * ldy : kBK * 2;
    if constexpr (DIR == S_LOGITS) {
      xrec -= kBK * 2;
      left -= kBK;
    }
    describe();
  }
  __device__ __forceinline__ void turn() {
    if (k != stop || slices <= 0) return;
    if (k == steps * kBK) {
      k = 0;
      ++pass;
    }
    find();
    // no scalar load may be under way where the paths meet: the reads of LDS there could not be told from it
    __builtin_amdgcn_s_waitcnt(kLdsDone);
  }

  template <int I> __device__ __forceinline__ void load(AR_LDS char* lds) {
    if constexpr (I < LX::kCount) load_lds(lds + (I * C::kThreads + wave * 64) * 16, x, lx.at(I, ldx, left));
    else load_lds(lds + C::kX + ((I - LX::kCount) * C::kThreads + wave * 64) * 16, y, ly.at(I - LX::kCount, ldy, kBK));
  }
};

// A wave's operands: a whole slice's of y, and a ring of x that is read kAhead products' rows ahead.
template <class C, int DIR> struct Operands {
  static constexpr int kRing = 4, kAhead = C::FM < kRing ? C::FM : kRing - 1;
  static_assert(2 * C::FM % kRing == 0, "two slices go round the ring");
  bf16x8 x[kRing], y[2][C::FN];
  int wm, wn, lane;
  template <int I, int SLOT> __device__ __forceinline__ void read_x(AR_LDS char* lds) {
    if constexpr (Stager<C, DIR>::kXAlong) x[SLOT % kRing] = read_along(lds, wm * C::MW + I * 16, lane);
    else x[SLOT % kRing] = read_across<C::BM>(lds, wm * C::MW + I * 16, lane);
  }
  template <int J, int SET> __device__ __forceinline__ void read_y(AR_LDS char* lds) {
    if constexpr (Stager<C, DIR>::kYAlong) y[SET][J] = read_along(lds + C::kX, wn * C::NW + J * 16, lane);
    else y[SET][J] = read_across<C::BN>(lds + C::kX, wn * C::NW + J * 16, lane);
  }
};

template <int I, int N, class F> __device__ __forceinline__ void each_of(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each_of<I + 1, N>(f);
  }
}

// The products of the slice in `here` (the SET-th of two), with the reads of the next one's y from `there`, of x a
// little ahead, and the loads of another slice into `to` between them, in this order: a wave issues in order, and a run
// of loads would hold its products up.
template <class C, int DIR, int SET> __device__ __forceinline__ void slice(Stager<C, DIR>& st, Operands<C, DIR>& o, AR_LDS char* here, AR_LDS char* there, AR_LDS char* to,
                                                                           f32x4 (&acc)[C::FM][C::FN]) {
  using O = Operands<C, DIR>;
  constexpr int kLoads = Stager<C, DIR>::kLoads, kEarly = C::FM * 3 / 4;  // the last of y have some products' time to return
  each_of<0, C::FM>([&](auto row) {
    constexpr int i = row, ahead = i + O::kAhead;
    each_of<kLoads * i / C::FM, kLoads * (i + 1) / C::FM>([&](auto l) { st.template load<l>(to); });
    if constexpr (i == C::FM - 1) st.advance();
    if constexpr (ahead < C::FM) o.template read_x<ahead, SET * C::FM + ahead>(here);
    else o.template read_x<ahead - C::FM, SET * C::FM + ahead>(there);
    if constexpr (i < kEarly) each_of<C::FN * i / kEarly, C::FN * (i + 1) / kEarly>([&](auto j) { o.template read_y<j, 1 - SET>(there); });
    each_of<0, C::FN>([&](auto j) {
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o.x[(SET * C::FM + i) % O::kRing], o.y[SET][j], acc[i][j], 0, 0, 0);
    });
    __builtin_amdgcn_sched_barrier(0);
  });
}

// Consecutive outputs of a row, of which `left` exist, at any address.
template <class E, class V> __device__ __forceinline__ void put(E* p, V v, int left) {
  constexpr int kN = sizeof(V) / sizeof(E);
  typedef E U __attribute__((ext_vector_type(kN), aligned(sizeof(E))));
  if (left >= kN) {
    *reinterpret_cast<U*>(p) = v;
  } else {
#pragma unroll
    for (int e = 0; e < kN - 1; ++e)
      if (e < left) p[e] = v[e];
  }
}

// Two products' registers, m 4 (lane / 16) on of 16 each, rounded and exchanged between the quarters of the wave: m
// 8 (lane / 16) on of the 32.
template <class V8, class V4> __device__ __forceinline__ V8 eight_of(f32x4 a, f32x4 b) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x2 x = __builtin_bit_cast(u32x2, __builtin_convertvector(a, V4)), y = __builtin_bit_cast(u32x2, __builtin_convertvector(b, V4));
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto p = __builtin_amdgcn_permlane32_swap(x[i], y[i], false, false);  // quarters (a0, a1, b0, b1) and (a2, a3, b2, b3)
    const auto q = __builtin_amdgcn_permlane16_swap(p[0], p[1], false, false);  // (a0, a2, b0, b2) and (a1, a3, b1, b3)
    r[i] = q[0];
    r[2 + i] = q[1];
  }
  return __builtin_bit_cast(V8, r);
}

// A barrier for what the workgroup leaves in LDS, which waits for no load or store of global memory.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(kLdsDone);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Shares of a product's depth: as many as give every compute unit a tile, by the rows that there are (12 tiles in 21
// shares run in one round where 32 took two; more shares are more partial sums to write and read).
__device__ __forceinline__ int splits_of(const Product& a, int nlen) {
  const int tiles = (nlen + a.bn - 1) / a.bn * a.mtiles;
  return tiles ? min(max(a.resident / tiles, 1), a.splits) : 1;
}

__device__ __forceinline__ const Counts& counts_of(const Product& a) { return reinterpret_cast<const Counts*>(a.pieces)[-1]; }
__device__ __forceinline__ int chunk_active(const Product& a) { return min(max(counts_of(a).active - a.chunk, 0), a.chunk_rows); }
// Rows of D, its second terms' among them.
__device__ __forceinline__ int d_rows(const Product& a, int active) { return active ? a.lo + active : 0; }

// Where a workgroup's tile t lies, and which slices of the depth it takes.
struct Place {
  int m0, n0, split, s0, s1;
};

// A wave's place in its workgroup.
struct Wave {
  int m, n, lane;
};

// What a logits tile's pick asks for: a lane's row's ids where they are few (row n of the wave's part for lane n), or
// the tile's entries and the first of them for the lane.
struct Own {
  typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
  i32x4 ids = {-1, -1, -1, -1};
  const uint32_t* entries = nullptr;
  int first = 0, end = 0;
};
template <class C> __device__ __forceinline__ Own own_of(const Product& a, const Place& at, int active, Wave wave) {
  Own own;
  const int n = at.n0 + wave.n * C::NW + wave.lane;
  if (a.ld_idt <= kFewIds) {
    if (wave.lane < C::NW && n < active) own.ids = *reinterpret_cast<const Own::i32x4*>(a.idt + int64_t(a.chunk + n) * kFewIds);
  } else {
    const int tile = (a.chunk + at.n0) / C::BN;
    const int32_t* at_m = a.starts + int64_t(tile) * (a.mtiles + 1) + at.m0 / C::BM;
    own.first = __builtin_amdgcn_readfirstlane(at_m[0]);
    own.end = __builtin_amdgcn_readfirstlane(at_m[1]);
    own.entries = a.entries + int64_t(tile) * a.entries_ld;
    if (own.first + wave.lane < own.end) own.ids[0] = int32_t(own.entries[own.first + wave.lane]);
  }
  return own;
}

// A logits tile: no logits where the piece has no rows (piece_left: those it has from the tile's first on), and the
// logits at the rows' own ids put away.
template <class C> __device__ __forceinline__ void pick_own(const Product& a, f32x4 (&acc)[C::FM][C::FN], const Place& at, const Own& own, int piece_left, Wave wave) {
  const int wm = wave.m, wn = wave.n, lane = wave.lane, wn0 = at.n0 + wn * C::NW;
  // Products stay as they are, without the temperature, until two of them have been subtracted: the difference to the
  // largest is exact next to it (its own is 0), where a rounding of 2^-24 of each logit would be one of the exponent
  // (one target's probability of 1 off by 1e-4 at logits of 1500; infinite exponentials from 2^26 on). Times a.scale,
  // whose rounding then is one of 2^-24 of the difference, it is the exponent of 2.
  if (piece_left < C::BM) {
    const int left = piece_left - wm * C::MW - lane / 16 * 4;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = i * 16 + e < left ? acc[i][j][e] : -INFINITY;
  }
  // the logits of the rows' own ids: every lane has one that may lie in the wave's part of the tile, and the wave
  // takes those that do one by one
  const auto pick = [&](uint32_t m, uint32_t n, uint32_t k) {
    const uint32_t r = m - wm * C::MW, c = n - wn * C::NW;
    for (uint64_t hit = __ballot(r < uint32_t(C::MW) && c < uint32_t(C::NW)); hit; hit &= hit - 1) {
      const int src = __builtin_ctzll(hit);
      const int row = __builtin_amdgcn_readlane(int(r), src), col = __builtin_amdgcn_readlane(int(c), src), which = __builtin_amdgcn_readlane(int(k), src);
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
        if (col / 16 == j) {
#pragma unroll
          for (int i = 0; i < C::FM; ++i)
            if (row / 16 == i) x = acc[i][j];
        }
      const float v = row % 4 == 0 ? x[0] : row % 4 == 1 ? x[1] : row % 4 == 2 ? x[2] : x[3];
      if (lane == row % 16 / 4 * 16 + col % 16) a.zt[int64_t(wn0 + col) * a.ld_idt + which] = v;
    }
  };
  if (a.ld_idt <= kFewIds) {
#pragma unroll 1
    for (int e = 0; e < kFewIds; ++e) {
      const int32_t id = e == 0 ? own.ids[0] : e == 1 ? own.ids[1] : e == 2 ? own.ids[2] : own.ids[3];
      pick(uint32_t(id - at.m0), id >= 0 ? uint32_t(wn * C::NW + lane) : ~0u, uint32_t(e));
    }
  } else {
#pragma unroll 1
    for (int e = own.first; e < own.end; e += 64) {
      const uint32_t x = e == own.first ? uint32_t(own.ids[0]) : e + lane < own.end ? own.entries[e + lane] : ~0u;
      pick(x == ~0u ? ~0u : x & 255, x >> 8 & 255, x >> 16);
    }
  }
}

// A bf16 call keeps its exponentials in fp16, as many bytes with eight times the precision: times kKept they are
// normal down to 2^-28 of the tile's largest, off by 2^-11 of their value or 2^-39 of the largest. (In bf16 D was
// rounded twice, and its products' results off by half as much again.)
constexpr float kKept = 16384;

// A logits tile's exponentials, largest values and sums. scratch: [2][WM][BN] of LDS.
template <class C, int KEEP> __device__ __forceinline__ void put_logits(const Product& a, f32x4 (&acc)[C::FM][C::FN], const Place& at, Wave wave, AR_LDS float* scratch) {
  static_assert(KEEP != D_BF16 || C::FM % 2 == 0, "bf16 is written by pairs of products");
  const int wm = wave.m, wn = wave.n, lane = wave.lane, wn0 = at.n0 + wn * C::NW, wm0 = at.m0 + wm * C::MW;
  AR_LDS float* top = scratch;  // [WM][BN]
  AR_LDS float* sum = top + C::WM * C::BN;  // [WM][BN]
  float mx[C::FN];
#pragma unroll
  for (int j = 0; j < C::FN; ++j) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2) m = fmaxf(fmaxf(m, acc[i][j][e]), acc[i][j][e + 1]);
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    if (lane < 16) top[wm * C::BN + wn * C::NW + j * 16 + lane] = m;
  }
  lds_barrier();
#pragma unroll
  for (int j = 0; j < C::FN; ++j) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < C::WM; ++w) m = fmaxf(m, top[w * C::BN + wn * C::NW + j * 16 + lane % 16]);
    mx[j] = m == -INFINITY ? 0.f : m;  // a tile without rows of the vocabulary: exponentials of 0
    float s = 0;
    const int64_t row = int64_t(wn0 + j * 16 + lane % 16) * a.Vp + wm0;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[i][j][e] = __builtin_amdgcn_exp2f((acc[i][j][e] - mx[j]) * a.scale);
        s += acc[i][j][e];
      }
      if constexpr (KEEP == D_BF16)
        if (i & 1) *reinterpret_cast<f16x8*>(reinterpret_cast<_Float16*>(a.d) + row + (i - 1) * 16 + lane / 16 * 8) = eight_of<f16x8, f16x4>(acc[i - 1][j] * kKept, acc[i][j] * kKept);
      if constexpr (KEEP == D_FP32) *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.part) + row + i * 16 + lane / 16 * 4) = acc[i][j];
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < 16) sum[wm * C::BN + wn * C::NW + j * 16 + lane] = s;
  }
  lds_barrier();
  if (wm == 0 && lane < 16)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int n = wn * C::NW + j * 16 + lane;
      float s = 0;
#pragma unroll
      for (int w = 0; w < C::WM; ++w) s += sum[w * C::BN + n];
      // a sum of 0 is a tile without a logit: its largest is no value that may pass the row's
      a.stats[int64_t(at.m0 / C::BM) * a.ld_stats + at.n0 + n] = float2{s == 0 ? -INFINITY : mx[j], s};
    }
}

// A gradient's tile, n < nlen of it.
template <class C, int DIR, int KEEP> __device__ __forceinline__ void put_gradient(const Product& a, f32x4 (&acc)[C::FM][C::FN], const Place& at, int nlen, Wave wave) {
  static_assert(KEEP != D_BF16 || C::FM % 2 == 0, "bf16 is written by pairs of products");
  const int lane = wave.lane, wn0 = at.n0 + wave.n * C::NW, wm0 = at.m0 + wave.m * C::MW;
  constexpr int kBytes = KEEP == D_BF16 ? 2 : 4;
  float factor = 1;
  if (!a.part) {
    // A scalar load (nothing writes there meanwhile), whose wait is not one for the next tile's slices; and waited for
    // here, for otherwise the compiler has the products' loop wait for it, and with it for all loads: 6% of d_hidden.
    typedef const __attribute__((address_space(4))) float* Constant;
    factor = *(Constant)(uintptr_t)&counts_of(a).factor;
    __builtin_amdgcn_s_waitcnt(kLdsDone);
  }
  // a tile of the vocabulary lies in one piece
  const Piece* p = nullptr;
  if constexpr (DIR == S_WEIGHT) p = a.pieces + __builtin_amdgcn_readfirstlane(piece_of<true>(a.pieces, a.P, at.n0));
#pragma unroll
  for (int j = 0; j < C::FN; ++j) {
    const int n = wn0 + j * 16 + lane % 16;
    char* row = nullptr;
    bool there = n < nlen;
    if (!a.part) {
      if constexpr (DIR == S_HIDDEN) {
        if (there) row = static_cast<char*>(a.dh) + int64_t(a.rows[a.chunk + n]) * a.dh_ld * kBytes;
      } else {
        there = n - p->start < p->rows;
        row = p->dw + int64_t(n - p->start) * p->dld * kBytes;
      }
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int m = wm0 + i * 16 + lane / 16 * 4;
      if (a.part) {
        if (there && m < a.Hp) {
          f32x4* q = reinterpret_cast<f32x4*>(a.part + at.split * a.part_stride + int64_t(n) * a.Hp + m);
          *q = a.accumulate ? *q + acc[i][j] : acc[i][j];
        }
      } else if constexpr (KEEP == D_BF16) {
        if (i & 1) {
          const int m8 = wm0 + (i - 1) * 16 + lane / 16 * 8;
          const bf16x8 v = eight_of<bf16x8, bf16x4>(acc[i - 1][j] * factor, acc[i][j] * factor);
          if (there && m8 < a.H) put(reinterpret_cast<__bf16*>(row) + m8, v, a.H - m8);
        }
      } else {
        if (there && m < a.H) put(reinterpret_cast<float*>(row) + m, acc[i][j] * factor, a.H - m);
      }
    }
  }
}

// KEEP: what a logits tile leaves behind: 0 only its sums, D_BF16 or D_FP32 the exponentials. The other directions:
// the outputs' type.
// Where tiles are many the matrix pipes are busy for 64-71% of the time at 8192 x 4096 x 128000, at the 1.8-1.9 GHz that
// power leaves, 1244-1321 TFLOP/s (on zeros, 2.3 GHz at the same share): the other third is what a SIMD's two waves
// wait for together, at the barrier of every slice. 256 x 256 outputs for 8 waves are
// what the accumulators hold: each slice's 32 KB are read into LDS for 4.2 MFLOP. With 64 deep double buffers the three
// took 7.8, 9.2 and 9.3 ms in place of 6.8, 6.4 and 7.0; in 32 x 32 x 16 products 2-8% more than in 16 x 16 x 32.
// Of up to 64 rows the reading of the output matrix bounds it: 8 x 2048 x 32000 in 25 us, 5.4 TB/s.
template <class C, int DIR, int KEEP> __global__ __launch_bounds__(C::kThreads, C::kWaves) void k_vocab_product(Product a) {
  __shared__ __attribute__((aligned(512))) char shared[C::kStages * C::kStage];
  using St = Stager<C, DIR>;
  using O = Operands<C, DIR>;
  constexpr int kLoads = St::kLoads;
  AR_LDS char *lds = (AR_LDS char*)shared, *last = lds + (C::kStages - 1) * C::kStage;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid / 64), wm = wave % C::WM, wn = wave / C::WM;
  const int active = DIR == S_LOGITS ? chunk_active(a) : d_rows(a, chunk_active(a));
  const int nlen = DIR == S_WEIGHT ? a.Vp : active;
  const uint32_t ntiles = (nlen + C::BN - 1) / C::BN, mtiles = a.mtiles, tiles = ntiles * mtiles, splits = splits_of(a, nlen), places = tiles * splits;
  const int depth = DIR == S_LOGITS ? a.Hp : DIR == S_HIDDEN ? a.Vp : (active + 2 * kBK - 1) / (2 * kBK) * 2 * kBK;
  const int steps = depth / kBK, all = steps * (a.planes == 1 ? 1 : 6);
  St st{a, 0, 0, tid, steps};
  st.wave = wave;
  const Wave w{wm, wn, lane};
  O o;
  o.wm = wm;
  o.wn = wn;
  o.lane = lane;

  const auto place = [&](uint32_t t) {
    Place p;
    p.split = int(t / tiles);
    // Workgroups go to the eight dies in turn: each die gets a run of tiles, and of a run eight tiles of n share
    // their m with the neighbours, so that both operands are found in the die's cache.
    uint32_t u = t - p.split * tiles;
    const uint32_t per = tiles / 8, more = tiles % 8, die = u % 8, i = u / 8;
    u = die * per + min(die, more) + i;
    const uint32_t group = u / (8 * mtiles), in_group = u - group * 8 * mtiles, width = min(8u, ntiles - group * 8);
    p.m0 = in_group / width * C::BM;
    p.n0 = (group * 8 + in_group % width) * C::BN;
    const int pairs = all / 2, share = pairs / splits, over = pairs % splits;
    p.s0 = (p.split * share + min(p.split, over)) * 2;
    p.s1 = p.s0 + (share + (p.split < over)) * 2;
    return p;
  };
  // The first kStages - 1 slices of a tile, on their way into LDS.
  const auto start = [&](const Place& p) {
    st.begin(p.m0, p.n0);
    if (p.s0 >= p.s1) return;
    st.seek(p.s0, p.s1);
    for (int i = 0; i < C::kStages - 1; ++i) {
      each_of<0, kLoads>([&](auto l) { st.template load<l>(lds + i * C::kStage); });
      st.advance();
      if (i & 1) st.turn();
    }
  };

  uint32_t t = blockIdx.x;
  if (t >= places) return;
  Place at = place(t);
  start(at);
  while (true) {
    Own own;
    if constexpr (DIR == S_LOGITS) own = own_of<C>(a, at, active, w);
    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // While a slice is multiplied, the next one's y (and the first of its x) are read from LDS and another is loaded
    // into LDS, kStages - 1 ahead, where the one before has been: one barrier a slice. Two at a time, for the two
    // sets of y.
    if (at.s0 < at.s1) {
      __builtin_amdgcn_s_waitcnt(waits((C::kStages - 2) * kLoads));
      __syncthreads();
      each_of<0, C::FN>([&](auto j) { o.template read_y<j, 0>(lds); });
      each_of<0, O::kAhead>([&](auto i) { o.template read_x<i, i>(lds); });
      AR_LDS char *to = last, *here = lds, *there = lds + C::kStage;
      const auto step = [&](auto set) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(waits((C::kStages - 3) * kLoads, false));  // this wave's loads of `there` have arrived
        __builtin_amdgcn_s_barrier();                                         // all waves' have, and `to` has been read
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        slice<C, DIR, set>(st, o, here, there, to, acc);
        to = here;
        here = there;
        there = there == last ? lds : there + C::kStage;
      };
      for (int s = at.s0; s < at.s1; s += 2) {
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        st.turn();
      }
    }
    __builtin_amdgcn_s_waitcnt(waits(0));
    __syncthreads();

    const int piece_left = DIR == S_LOGITS ? st.rows - (at.m0 - st.start) : 0;  // rows of the piece from the tile's first on
    if constexpr (DIR == S_LOGITS) pick_own<C>(a, acc, at, own, piece_left, w);

    // The next tile's first slices travel while this one's results are written; `last` is free of them until the
    // next tile's first barrier.
    const Place done = at;
    t += gridDim.x;
    const bool more = t < places;
    if (more) {
      at = place(t);
      start(at);
    }

    if constexpr (DIR == S_LOGITS) put_logits<C, KEEP>(a, acc, done, w, (AR_LDS float*)last);
    else put_gradient<C, DIR, KEEP>(a, acc, done, nlen, w);
    if (!more) return;
  }
}

// Few rows against an output matrix that loads into LDS cannot bring as bf16 (fp32, or rows at odd addresses): the
// products read it as it is, split it into terms on the way to LDS and multiply all terms of a slice at once, where
// many rows are better served by a copy (which reads, writes and reads again what is read once here). S_LOGITS and
// S_HIDDEN only: the output matrix is X. (us a loss of 2048 x 32000, so and with a copy: fp32 of 8 rows 77 and 292, of 64
// 92 and 294; bf16 of 64 rows of odd width 49 and 86.) kDeep slices are on their way in registers. PARTS: sixteen rows
// each, of which products are formed.
constexpr int kFewRows = 64, kDeep = 3;
template <int DT, int DIR, int KEEP, int PARTS> __global__ __launch_bounds__(TileF<DT>::kThreads, TileF<DT>::kWaves) void k_vocab_few(Product a) {
  using C = TileF<DT>;
  static_assert(C::WN == 1 && C::BN == 64 && C::kThreads == 256, "the loads below");
  constexpr bool kAlong = DIR == S_LOGITS;
  // terms of X and of Y; elements of a 16-byte load
  constexpr int PL = DT == D_FP32 ? 3 : 1, PY = DT == D_BF16 && !kAlong ? 2 : PL, kPer = DT == D_FP32 ? 4 : 8;
  constexpr int kLoads = C::BM * kBK / kPer / C::kThreads, kRow = (kAlong ? kBK : C::BM) / kPer;
  constexpr int kSlice = PL * C::kX + PY * C::kY;
  using E = std::conditional_t<DT == D_FP32, float, uint16_t>;
  typedef E V __attribute__((ext_vector_type(kPer)));
  // (in global memory: a load that may be of LDS would be waited for with it)
  typedef E Any __attribute__((ext_vector_type(kPer), aligned(sizeof(E)), address_space(1)));
  typedef E Global __attribute__((address_space(1)));
  constexpr int kCols = kAlong ? kBK : C::BM;
  __shared__ __attribute__((aligned(512))) char shared[2 * kSlice];
  AR_LDS char* lds = (AR_LDS char*)shared;
  const int tid = threadIdx.x, lane = tid & 63, wm = __builtin_amdgcn_readfirstlane(tid / 64);
  const Wave w{wm, 0, lane};
  const int active = chunk_active(a), steps = (DIR == S_LOGITS ? a.Hp : a.Vp) / kBK;
  const int ntiles = (active + C::BN - 1) / C::BN, tiles = ntiles * a.mtiles;
  struct Slice {
    V x[kLoads];
    bf16x8 y[PY];
  };
  const int splits = splits_of(a, active);
  for (int t = blockIdx.x; t < tiles * splits; t += gridDim.x) {
    const int split = t / tiles, u = t - split * tiles, share = steps / splits, over = steps % splits;
    const int s0 = split * share + min(split, over);
    const Place at{u / ntiles * C::BM, u % ntiles * C::BN, split, s0, s0 + share + (split < over)};
    int rows = 0, start = 0, next = 0;
    int64_t ld = 0;
    uintptr_t wp = 0;
    const auto take_at = [&](int32_t row) {
      const int p = __builtin_amdgcn_readfirstlane(piece_of<true>(a.pieces, a.P, row));
      wp = uintptr_t(uniform(reinterpret_cast<int64_t>(a.pieces[p].w)));
      ld = uniform(a.pieces[p].ld);
      rows = __builtin_amdgcn_readfirstlane(a.pieces[p].rows);
      start = __builtin_amdgcn_readfirstlane(a.pieces[p].start);
      next = p + 1 < a.P ? __builtin_amdgcn_readfirstlane(a.pieces[p + 1].start) : 0x7fffffff;
    };
    if constexpr (kAlong) take_at(at.m0);
    Own own;
    if constexpr (kAlong) own = own_of<C>(a, at, active, w);

    // Every load is of memory that is there, so that none depends on another's branch: behind the piece's rows its last
    // one is read (logits without a row, and rows that meet zeros of D), behind a row's end its last elements, which
    // store() moves to their places, and behind the last slice that one again.
    const auto load = [&](Slice& r, int s) {
      const int k = min(s, at.s1 - 1) * kBK;
      if (!kAlong && (k < start || k >= next)) take_at(k);
      const int row0 = kAlong ? at.m0 - start : k - start, col0 = kAlong ? k : at.m0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int q = i * C::kThreads + tid;
        r.x[i] = *reinterpret_cast<const Any*>(reinterpret_cast<const Global*>(wp) + int64_t(min(row0 + q / kRow, rows - 1)) * ld + min(col0 + q % kRow * kPer, a.H - kPer));
      }
      const int64_t n = min(at.n0 + tid / 4, active - 1);
      const char* p = (DIR == S_LOGITS ? a.hp + (a.chunk + n) * PL * a.Hp * 2 : a.d + n * PL * a.Vp * 2) + (k + tid % 4 * 8) * 2;
#pragma unroll
      for (int i = 0; i < PY; ++i)
        r.y[i] = *reinterpret_cast<const __attribute__((address_space(1))) bf16x8*>(reinterpret_cast<uintptr_t>(p) + int64_t(i) * (kAlong ? a.Hp : PY == 2 ? a.lo * int64_t(a.Vp) : a.Vp) * 2);
    };
    const auto store = [&](Slice& r, int s, AR_LDS char* to) {
      const int col0 = kAlong ? s * kBK : at.m0;
      if (col0 + kCols > a.H) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int over = max(col0 + (i * C::kThreads + tid) % kRow * kPer - (a.H - kPer), 0);  // how far the load lies before its place
          V v = {};
#pragma unroll
          for (int d = 0; d < kPer; ++d)
#pragma unroll
            for (int j = 0; j + d < kPer; ++j) v[j] = over == d ? r.x[i][j + d] : v[j];
          r.x[i] = v;
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t q = i * C::kThreads + tid, outer = q / kRow, byte = q % kRow * kPer * 2;  // byte of the row in a term's slice
        AR_LDS char* p = to + (kAlong ? outer * 64 + ((byte / 16) ^ along_swizzle(outer)) * 16 + byte % 16
                                      : outer * (C::BM * 2) + ((byte / 32) ^ across_swizzle<C::BM>(outer)) * 32 + byte % 32);
        if constexpr (DT == D_BF16) {
          *reinterpret_cast<AR_LDS V*>(p) = r.x[i];
        } else {
          bf16x4 o[3];
          split3_of<4>(r.x[i], o);
#pragma unroll
          for (int l = 0; l < 3; ++l) *reinterpret_cast<AR_LDS bf16x4*>(p + l * C::kX) = o[l];
        }
      }
#pragma unroll
      for (int i = 0; i < PY; ++i) {
        const uint32_t row = tid / 4;
        *reinterpret_cast<AR_LDS bf16x8*>(to + PL * C::kX + i * C::kY + row * 64 + ((tid % 4) ^ along_swizzle(row)) * 16) = r.y[i];
      }
    };

    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    Slice r[kDeep];
    if (at.s0 < at.s1) {
#pragma unroll
      for (int i = 0; i < kDeep; ++i) load(r[i], at.s0 + i);
    }
    for (int s = at.s0; s < at.s1; s += kDeep) {
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        if (s + i >= at.s1) break;
        AR_LDS char* here = lds + ((s - at.s0 + i) & 1) * kSlice;
        store(r[i], s + i, here);
        load(r[i], s + i + kDeep);
        lds_barrier();  // the slice is there, and the one before the last has been multiplied
        bf16x8 y[PY][PARTS];
#pragma unroll
        for (int l = 0; l < PY; ++l)
#pragma unroll
          for (int j = 0; j < PARTS; ++j) y[l][j] = read_along(here + PL * C::kX + l * C::kY, j * 16, lane);
#pragma unroll
        for (int f = 0; f < C::FM; ++f) {
          bf16x8 x[PL];
#pragma unroll
          for (int l = 0; l < PL; ++l) {
            if constexpr (kAlong) x[l] = read_along(here + l * C::kX, wm * C::MW + f * 16, lane);
            else x[l] = read_across<C::BM>(here + l * C::kX, wm * C::MW + f * 16, lane);
          }
#pragma unroll
          for (int pass = 0; pass < (PL == 3 ? 6 : PY); ++pass)
#pragma unroll
            for (int j = 0; j < PARTS; ++j)
              acc[f][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[plane_x(pass, PL)], y[PY == 2 ? 1 - pass : plane_y(pass, PL)][j], acc[f][j], 0, 0, 0);
        }
      }
    }
    __syncthreads();
    if constexpr (kAlong) {
      pick_own<C>(a, acc, at, own, rows - (at.m0 - start), w);
      put_logits<C, KEEP>(a, acc, at, w, (AR_LDS float*)lds);
      __syncthreads();
    } else {
      put_gradient<C, DIR, KEEP>(a, acc, at, active, w);
    }
  }
}

// ----------------------------------------------------------------------------
// softmax statistics, D, losses
// ----------------------------------------------------------------------------
struct Soft {
  Counts* counts;
  const int32_t* rows;
  const float* weights;
  const float2* stats;
  int64_t ld_stats;
  int32_t blocks, chunk, chunk_rows, reduction;
  int32_t planes, block;  // block: columns a statistic covers
  int64_t Vp;
  float scale;  // log2(e) / temperature
  float2* lse;   // [chunk rows] in two parts: the largest product, the log of the sum around it (their sum would round
                 // p by 2^-24 of the logit)
  float* coef;   // [chunk rows]: the row's weight times Counts::share; 0 behind the rows
  float* exps;   // fp32: exp(z - m)
  char* d;
  int32_t lo;    // as in Product
};

// What the rows' own ids are for.
struct Ends {
  const float2* teacher;  // by original row
  const int32_t* idt;
  int32_t ld_idt;
  const float* zt;
  float* row_loss;  // [rows that take part], weighted
  float* each;      // by original row, or null
  float* total;     // or null
};

// The teacher's probability of a row's entry (1 for the one target), and x = its logit less the row's largest, over
// the temperature.
struct Teacher {
  const Targets& t;
  int64_t row;
  float2 stat;
  __device__ __forceinline__ float q(int k, float* x) const {
    *x = 0;
    if (!t.K) return 1.f;
    *x = (logit_at(t.logits, t.logits_dtype, row * t.logits_ld + k) - stat.x) / t.temperature;
    return expf(*x) / stat.y;
  }
};
__device__ __forceinline__ Teacher teacher_of(const Targets& t, const Ends& e, int64_t row) { return Teacher{t, row, t.K ? e.teacher[row] : float2{0, 1}}; }

// The rows' softmax statistics, weights and losses, 16 rows a workgroup: first a wave's lanes are 16 rows x 4
// statistics, and its 16 waves share the statistics; then each wave takes a row's ids. 8192 rows x 500 statistics: 25
// us; few rows take 4, a chain of waits for memory.
constexpr int kJoinThreads = 1024, kJoinRows = 16;
__global__ __launch_bounds__(kJoinThreads) void k_vocab_join(Soft a, Ends e, Targets t) {
  __shared__ float2 part[kJoinThreads / 64][kJoinRows];
  __shared__ float2 row_lse[kJoinRows];
  const int row = threadIdx.x % 16, slice = threadIdx.x / 16, wave = threadIdx.x / 64, lane = threadIdx.x & 63;
  const int active = min(max(a.counts->active - a.chunk, 0), a.chunk_rows), end = (active + kUnit - 1) / kUnit * kUnit;
  for (int r0 = blockIdx.x * kJoinRows; r0 < end; r0 += gridDim.x * kJoinRows) {
    const int r = r0 + row;
    float m = -INFINITY, s = 0;
    const auto join = [&](float& m, float& s, float om, float os) {
      if (os == 0) return;
      const float top = fmaxf(m, om);  // a NaN sum stays one
      s = (m == top ? s : s * exp2f((m - top) * a.scale)) + (om == top ? os : os * exp2f((om - top) * a.scale));
      m = top;
    };
    const auto join_lanes = [&](float& m, float& s) {
#pragma unroll
      for (int d = 16; d < 64; d <<= 1) {
        const float om = __shfl_xor(m, d), os = __shfl_xor(s, d);
        // in the lanes' order, so that both partners get the same
        float lm = lane & d ? om : m, ls = lane & d ? os : s;
        join(lm, ls, lane & d ? m : om, lane & d ? s : os);
        m = lm;
        s = ls;
      }
    };
    if (r < active)
      for (int b = slice; b < a.blocks; b += kJoinThreads / 16) {
        const float2 x = a.stats[int64_t(b) * a.ld_stats + r];
        join(m, s, x.x, x.y);
      }
    join_lanes(m, s);
    if (lane < 16) part[wave][row] = float2{m, s};
    __syncthreads();
    if (wave == 0) {
      m = -INFINITY, s = 0;
      for (int w = lane / 16; w < kJoinThreads / 64; w += 4) join(m, s, part[w][row].x, part[w][row].y);
      join_lanes(m, s);
      float2 lse = {0, 0};
      float coef = 0;
      if (r < active) {
        lse = float2{m, log2f(s)};
        // in 64 bits: a weight over a small temperature may pass the largest fp32 value where its share of the mean does not
        coef = float((a.weights ? double(a.weights[a.rows[a.chunk + r]]) : 1.) * a.counts->share);
      }
      if (lane < 16) {
        a.lse[r] = row_lse[row] = lse;
        a.coef[r] = coef;
      }
    }
    __syncthreads();
    const int i = r0 + wave;
    if (i < active) {
      const int64_t from = a.rows[a.chunk + i];
      const Teacher teacher = teacher_of(t, e, from);
      float loss = 0;
      for (int k = lane; k < e.ld_idt; k += 64) {
        if (e.idt[(a.chunk + i) * int64_t(e.ld_idt) + k] < 0) continue;
        float x;
        const float q = teacher.q(k, &x);
        if (q != 0) loss += q * ((t.K ? x - logf(teacher.stat.y) : 0.f) + ((row_lse[wave].x - e.zt[int64_t(i) * e.ld_idt + k]) * a.scale + row_lse[wave].y) * kLn2);
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) loss += __shfl_xor(loss, d);
      if (lane == 0) {
        if (a.weights) loss *= a.weights[from];
        if (e.each) e.each[from] = loss;
        else e.row_loss[a.chunk + i] = loss;
      }
    }
    __syncthreads();
  }
}

// The call's loss from its rows' (of launches before): one workgroup adds them up, in 64 bits and in an order that their
// number fixes: beside the normalizing pass, or in 2 to 5 us behind the join (whose last workgroup, known by a counter, took a
// call no less time).
constexpr int kNormThreads = 256;
__device__ __forceinline__ void put_total(const Soft& a, const Ends& e) {
  __shared__ double wave_sum[kNormThreads / 64];
  const int active = a.counts->active, lane = threadIdx.x & 63;
  double sum = 0;
  constexpr int kTogether = 16;  // on their way at once: behind the last row that one again, for nothing
  for (int64_t i0 = threadIdx.x; i0 < active; i0 += kTogether * kNormThreads) {
    float x[kTogether];
#pragma unroll
    for (int q = 0; q < kTogether; ++q) x[q] = e.row_loss[min(i0 + q * kNormThreads, int64_t(active) - 1)];
#pragma unroll
    for (int q = 0; q < kTogether; ++q) sum += i0 + q * kNormThreads < active ? x[q] : 0.f;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_down(sum, d);
  if (lane == 0) wave_sum[threadIdx.x / 64] = sum;
  __syncthreads();
  if (threadIdx.x) return;
  sum = 0;
  for (int w = 0; w < kNormThreads / 64; ++w) sum += wave_sum[w];
  if (a.reduction == R_MEAN && a.counts->mean) sum /= a.counts->mean;
  *e.total = a.counts->bad ? NAN : float(sum);
}
__global__ __launch_bounds__(kNormThreads) void k_vocab_total(Soft a, Ends e) { put_total(a, e); }

// D at an id of a row: c (p - q), q the sum over the row's equal ids.
template <int DT> __device__ __forceinline__ void put_own(const Soft& a, const Ends& e, int i, int k, int32_t id, float q) {
  const float d = a.coef[i] * (exp2f((e.zt[int64_t(i) * e.ld_idt + k] - a.lse[i].x) * a.scale - a.lse[i].y) - q);
  __bf16* row = reinterpret_cast<__bf16*>(a.d) + int64_t(i) * (DT == D_BF16 ? 1 : 3) * a.Vp;
  if constexpr (DT == D_BF16) {
    row[id] = __bf16(d);
    if (a.lo) row[a.lo * a.Vp + id] = __bf16(d - float(__bf16(d)));
  } else {
    __bf16 b[3];
    split3(d, b);
#pragma unroll
    for (int j = 0; j < 3; ++j) row[j * a.Vp + id] = b[j];
  }
}

// exp(z - m) -> c p (c but for Counts::factor), in place for bf16, 16 rows x 512 columns a workgroup: every statistic's factor once, then 16 bytes a lane.
// Bound by memory: 8192 x 128000 in bf16, 2.1 GB each way, take 744 us, 5.7 TB/s.
constexpr int kNormRows = 16, kNormCols = 512, kBatch = 4;
template <int DT> __global__ __launch_bounds__(kNormThreads) void k_vocab_normalize(Soft a, Ends e, Targets t) {
  if (e.total && blockIdx.x + 1 == gridDim.x) put_total(a, e);
  constexpr int kBlocks = kNormCols / 64;  // no statistic covers fewer columns
  __shared__ float factor[kNormRows][kBlocks];
  const int active = min(max(a.counts->active - a.chunk, 0), a.chunk_rows);
  const int end = (a.lo && active ? a.lo : (active + 2 * kBK - 1) / (2 * kBK) * 2 * kBK) / kNormRows;
  const int64_t cols = (a.Vp + kNormCols - 1) / kNormCols, tiles = cols * end;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int r0 = int(tile / cols) * kNormRows;
    const int64_t c0 = (tile % cols) * kNormCols;
    static_assert(kNormThreads >= kNormRows * kFewIds, "a thread for each of a tile's few ids");
    const int own_row = r0 + threadIdx.x / kFewIds, own_k = threadIdx.x % kFewIds;
    const int32_t own = e.ld_idt == kFewIds && threadIdx.x < kNormRows * kFewIds && own_row < active ? e.idt[int64_t(a.chunk + own_row) * kFewIds + own_k] : -1;
    {
      const int r = threadIdx.x % kNormRows, b = threadIdx.x / kNormRows;
      const int64_t c = c0 + b * 64;
      float f = 0;
      const float w = b < kBlocks ? a.coef[r0 + r] : 0.f;
      if (w != 0 && c < a.Vp) f = exp2f((a.stats[c / a.block * a.ld_stats + r0 + r].x - a.lse[r0 + r].x) * a.scale - a.lse[r0 + r].y) * w;
      if (b < kBlocks) factor[r][b] = DT == D_BF16 ? f / kKept : f;
    }
    __syncthreads();
    constexpr int kLanes = kNormCols / 8;
    const int c8 = threadIdx.x % kLanes * 8;
    if (c0 + c8 < a.Vp)
      for (int r4 = threadIdx.x / kLanes; r4 < kNormRows; r4 += kBatch * kNormThreads / kLanes) {
        using In = std::conditional_t<DT == D_BF16, f16x8, f32x8>;
        In v[kBatch];  // loaded together
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int r = r4 + q * kNormThreads / kLanes;
          v[q] = In{};
          if (r0 + r >= active) continue;
          if constexpr (DT == D_BF16) v[q] = *reinterpret_cast<const In*>(reinterpret_cast<const _Float16*>(a.d) + int64_t(r0 + r) * a.Vp + c0 + c8);
          else v[q] = *reinterpret_cast<const In*>(a.exps + int64_t(r0 + r) * a.Vp + c0 + c8);
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int r = r4 + q * kNormThreads / kLanes;
          const float f = factor[r][c8 / 64];
          if constexpr (DT == D_BF16) {
            bf16x8 o, o2;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float d = float(v[q][j]) * f;  // (a second term only few rows keep)
              o[j] = __bf16(d);
              o2[j] = __bf16(d - float(o[j]));
            }
            __bf16* to = reinterpret_cast<__bf16*>(a.d) + int64_t(r0 + r) * a.Vp + c0 + c8;
            *reinterpret_cast<bf16x8*>(to) = o;
            if (a.lo) *reinterpret_cast<bf16x8*>(to + a.lo * a.Vp) = o2;
          } else {
            bf16x8 o[3];
            split3_of<8>(v[q] * f, o);
#pragma unroll
            for (int i = 0; i < 3; ++i)
              *reinterpret_cast<bf16x8*>(reinterpret_cast<__bf16*>(a.d) + (int64_t(r0 + r) * 3 + i) * a.Vp + c0 + c8) = o[i];
          }
        }
      }
    __syncthreads();
    if (own >= c0 && own < c0 + kNormCols) {
      const Teacher teacher = teacher_of(t, e, a.rows[a.chunk + own_row]);
      float q = 0, x;
      for (int l = 0; l < kFewIds; ++l)
        if (e.idt[int64_t(a.chunk + own_row) * kFewIds + l] == own) q += teacher.q(l, &x);
      put_own<DT>(a, e, own_row, own_k, own, q);
    }
  }
}

// More ids a row than kFewIds: a wave for 64 of a row's, which it compares with all of the row's, 64 in registers.
template <int DT> __global__ __launch_bounds__(256) void k_vocab_own(Soft a, Ends e, Targets t) {
  const int active = min(max(a.counts->active - a.chunk, 0), a.chunk_rows), lane = threadIdx.x & 63, parts = (e.ld_idt + 63) / 64;
  for (int64_t n = int64_t(blockIdx.x) * 4 + threadIdx.x / 64; n < int64_t(active) * parts; n += int64_t(gridDim.x) * 4) {
    const int i = int(n / parts), k = int(n % parts) * 64 + lane;
    const int32_t* ids = e.idt + (a.chunk + i) * int64_t(e.ld_idt);
    const Teacher teacher = teacher_of(t, e, a.rows[a.chunk + i]);
    const int32_t id = k < e.ld_idt ? ids[k] : -1;
    float sum = 0;
    for (int l0 = 0; l0 < e.ld_idt; l0 += 64) {
      const int32_t other = l0 + lane < e.ld_idt ? ids[l0 + lane] : -1;
      float x, q = 0;
      if (other >= 0) q = teacher.q(l0 + lane, &x);
      for (int l = 0; l < min(64, e.ld_idt - l0); ++l) {
        const float ql = as_f(__builtin_amdgcn_readlane(as_u(q), l));
        sum += __builtin_amdgcn_readlane(other, l) == id ? ql : 0.f;
      }
    }
    if (id >= 0) put_own<DT>(a, e, i, k, id, sum);
  }
}

// Partial gradients [splits][n][Hp] joined in order, into the outputs. Bound by memory: 67 MB into 8 in 14 us, 5.3 TB/s.
template <int DIR, int DT> __global__ __launch_bounds__(256) void k_vocab_sum(Product a) {
  const int n_end = DIR == S_WEIGHT ? a.Vp : chunk_active(a), per = a.Hp / 4, lo = DIR == S_HIDDEN ? a.lo : 0;
  const int64_t all = int64_t(n_end) * per;
  const int splits = splits_of(a, DIR == S_WEIGHT ? n_end : d_rows(a, n_end));
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 256) {
    const int n = int(i / per), m = int(i % per) * 4;
    if (m >= a.H) continue;
    char* row;
    constexpr int e = DT == D_BF16 ? 2 : 4;
    if constexpr (DIR == S_HIDDEN) {
      row = static_cast<char*>(a.dh) + int64_t(a.rows[a.chunk + n]) * a.dh_ld * e;
    } else {
      const Piece& p = a.pieces[piece_of<true>(a.pieces, a.P, n)];
      if (n - p.start >= p.rows) continue;
      row = p.dw + int64_t(n - p.start) * p.dld * e;
    }
    f32x4 s = {0, 0, 0, 0};
    const auto add = [&](const float* from) {
      int k = 0;
      for (; k + 8 <= splits; k += 8) {  // eight on their way together, added in order
        f32x4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = *reinterpret_cast<const f32x4*>(from + (k + q) * a.part_stride);
#pragma unroll
        for (int q = 0; q < 8; ++q) s += v[q];
      }
      for (; k < splits; ++k) s += *reinterpret_cast<const f32x4*>(from + k * a.part_stride);
    };
    if (lo) add(a.part + int64_t(lo + n) * a.Hp + m);
    add(a.part + int64_t(n) * a.Hp + m);
    s *= counts_of(a).factor;
    if constexpr (DT == D_BF16) put(reinterpret_cast<__bf16*>(row) + m, __builtin_convertvector(s, bf16x4), a.H - m);
    else put(reinterpret_cast<float*>(row) + m, s, a.H - m);
  }
}

// ----------------------------------------------------------------------------
// host
// ----------------------------------------------------------------------------
size_t up(size_t n, size_t unit = 256) { return (n + unit - 1) / unit * unit; }
// Workgroups of a launch: a dispatch's work-items are a 32-bit number, and some workgroups have 1024.
int64_t blocks_of(int64_t n) { return std::max<int64_t>(1, std::min<int64_t>(n, std::min<int64_t>(launch_blocks(), int64_t(1) << 21))); }

enum Size { Z_S = 0, Z_M = 1, Z_L = 2, Z_F = 3 };

// Scratch that one chunk of tokens may take (plan_of).
constexpr int64_t kChunkBytes = int64_t(4) << 30;
constexpr int kUnits = 256;  // compute units
// Hidden elements that the first launch's one workgroup packs itself rather than leaving them to another launch.
// (us a loss, so and with the launch: 16 x 64 fp32 26.7 and 26.6, 8 x 2048 bf16 45.7 and 41.8, 48 x 256 31.6 and 26.8.)
constexpr int64_t kFewElements = 4096;

struct Plan {
  int planes, Hp, Kp;  // Kp: ids of a row, whole vectors of them
  int64_t V = 0, Vp = 0, Tpad, Tc, chunks;
  bool packed;  // the output matrix is copied as bf16 terms
  bool few;     // or split on its way into few rows' products
  int lo;       // D is two bf16 terms, the second ones from this row on; or 0
  Size logits, hidden, weight;
  int hidden_splits = 1, weight_splits = 1;
  bool hidden_part = false;  // d_hidden's products leave partial sums
  int block;  // columns a statistic covers: a logits tile's
  int tile_rows;  // rows of a logits tile
  // offsets in the workspace
  size_t counts, pieces, rows, flags, teacher, idt, hp, wp, lse, coef, row_loss, zt, starts, entries, stats, exps, d, part, bytes;
};

int64_t tiles_of(Size z, int64_t m, int64_t n) {
  const int64_t bm = z == Z_L ? 256 : z == Z_F ? 64 : 128, bn = z == Z_L ? 256 : z == Z_M ? 128 : 64;
  return ((m + bm - 1) / bm) * ((n + bn - 1) / bn);
}

// Large tiles read each operand half as often as middle ones, but where they are half empty, or fewer than the compute
// units, the middle ones win (us a bf16 loss of width 2048 in large and in middle tiles: 100 rows x 98304 168 and 125;
// 256 rows x 16384, 64 large tiles, 67 and 47, x 32768 70 and 66, x 49152, 192 of them, 73 and 83, x 98304 154 and 174).
Size size_for(int64_t m, int64_t n, int64_t splits) {
  if (n <= kFewRows) return Z_S;
  if (n <= 128) return Z_M;
  return tiles_of(Z_L, m, n) * splits >= kUnits * 3 / 4 ? Z_L : Z_M;
}

// How often a product's depth is split so that its tiles fill the device (us a call with gradients, so and unsplit:
// 8 x 2048 x 32000 117 and 287, 1024 x 1024 x 32000 271 and 796, 48 x 256 x 1000 47 and 54).
int splits_for(int64_t tiles, int64_t steps, int64_t part_bytes) {
  const int64_t want = (2 * kUnits) / std::max<int64_t>(tiles, 1), most = std::min<int64_t>(steps / 4, (int64_t(256) << 20) / std::max<int64_t>(part_bytes, 1));
  return int(std::max<int64_t>(1, std::min(want, most)));
}

Plan plan_of(const Vocab& v, bool grad) {
  Plan p{};
  p.planes = v.dtype == D_FP32 ? 3 : 1;
  p.Hp = int(up(size_t(v.H), 2 * kBK));
  p.Kp = int(up(size_t(std::max(1, v.top)), 4));
  p.packed = v.dtype == D_FP32 || v.H % 8;
  for (const VocabPiece& q : v.pieces) {
    p.V += q.rows;
    p.Vp += int64_t(up(size_t(q.rows), kUnit));
    if (reinterpret_cast<uintptr_t>(q.w) % 16 || q.ld % 8 || q.ld >= (1 << 21)) p.packed = true;
  }
  p.few = p.packed && v.T <= kFewRows && v.H >= 8;  // (a whole vector in every row)
  if (p.few) p.packed = false;
  // Few rows of bf16 keep D as two terms: a result has few terms there, whose roundings do not even out. As one bf16 value
  // D left bf16 gradients of up to 128 rows as much as 2.2 times as far from 64 bits as an fp32 D does, of 129 and more 1.1
  // to 1.6 times; as two, 1.00 times. The second terms are more rows of D (and the hidden rows are there twice), so that
  // W is read once: us a call with gradients, so and with one term, 8 x 2048 x 32000 119 and 115, 48 x 256 x 1000 46.4
  // and 43.7, 64 x 2048 x 32000 145 and 120. (100 x 2048 x 32000 took 195 and 147: more rows keep one.)
  p.lo = grad && v.dtype == D_BF16 && v.T <= kFewRows ? (v.T <= 32 ? 32 : 64) : 0;
  p.Tpad = int64_t(up(size_t(std::max<int64_t>(v.T, 1)), kUnit));
  // a chunk's scratch: statistics at their finest, the own ids' logits, log-sum-exp and weight, and with gradients the
  // exponentials and D
  const int64_t per = p.Vp / 64 * 8 + p.Kp * 4 + 12 + (grad ? (v.dtype == D_FP32 ? 10 : 2) * p.Vp : 0);
  p.Tc = std::min(p.Tpad, std::max<int64_t>(kUnit, kChunkBytes / per / kUnit * kUnit));
  p.chunks = (p.Tpad + p.Tc - 1) / p.Tc;
  const int64_t n = std::min(p.Tc, v.T), passes = p.planes == 1 ? 1 : 6;
  p.logits = size_for(p.Vp, n, 1);
  const Size few = v.dtype == D_FP32 ? Z_F : Z_S;
  if (p.few) p.logits = few;
  p.block = p.logits == Z_L ? 256 : p.logits == Z_F ? 64 : 128;
  p.tile_rows = p.logits == Z_L ? 256 : p.logits == Z_M ? 128 : 64;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += up(bytes); return o; };
  static_assert(sizeof(Counts) % alignof(Piece) == 0, "the pieces follow");
  p.counts = take(sizeof(Counts) + sizeof(Piece) * v.pieces.size());
  p.pieces = p.counts + sizeof(Counts);
  p.rows = take(size_t(p.Tpad) * 4);
  p.flags = take(size_t(p.Tpad));
  p.teacher = take(v.top ? size_t(p.Tpad) * 8 : 0);
  p.idt = take(size_t(p.Kp) * size_t(p.Tpad) * 4);
  p.hp = take(size_t(p.Tpad) * size_t(p.planes) * size_t(p.Hp) * 2);
  p.wp = take(p.packed ? size_t(p.Vp) * size_t(p.planes) * size_t(p.Hp) * 2 : 0);
  p.lse = take(size_t(p.Tc) * 8);
  p.coef = take(size_t(p.Tc) * 4);
  p.row_loss = take(size_t(p.Tpad) * 4);
  p.zt = take(size_t(p.Tc) * size_t(p.Kp) * 4);
  const bool sorted = p.Kp > kFewIds;
  p.starts = take(sorted ? size_t(p.Tpad / p.tile_rows) * size_t(p.Vp / p.block + 1) * 4 : 0);
  p.entries = take(sorted ? size_t(p.Tpad) * size_t(p.Kp) * 4 : 0);
  p.stats = take(size_t(p.Vp / p.block) * size_t(p.Tc) * 8);
  if (grad) {
    p.exps = take(v.dtype == D_FP32 ? size_t(p.Tc) * size_t(p.Vp) * 4 : 0);
    p.d = take(size_t(p.Tc) * size_t(p.Vp) * size_t(p.planes) * 2);
    const int64_t hidden_steps = p.Vp / kBK * (p.few ? 1 : passes);
    const int64_t nd = p.lo && !p.few ? 2 * p.lo : n;
    p.hidden = p.few ? few : size_for(v.H, nd, hidden_steps / 8);
    p.hidden_splits = splits_for(tiles_of(p.hidden, v.H, nd), hidden_steps, nd * p.Hp * 4);
    p.hidden_part = p.hidden_splits > 1 || (p.lo && !p.few);
    p.weight = size_for(v.H, p.Vp, 1);
    if (p.chunks == 1) p.weight_splits = splits_for(tiles_of(p.weight, v.H, p.Vp), ((p.lo ? 2 * p.lo : n) + kBK - 1) / kBK * passes, p.Vp * p.Hp * 4);
    const size_t dh = p.hidden_part ? size_t(p.hidden_splits) * size_t(p.Tc) * size_t(p.Hp) * 4 : 0;
    const size_t dw = p.weight_splits > 1 || p.chunks > 1 ? size_t(p.weight_splits) * size_t(p.Vp) * size_t(p.Hp) * 4 : 0;
    p.part = take(p.chunks > 1 ? dh + dw : std::max(dh, dw));  // chunks add to dW's across dh's
  }
  p.bytes = at;
  return p;
}

template <int DT, int DIR, int KEEP> void launch_product(Sequence& s, const Plan& p, Size z, int64_t tiles, Product a) {
  const int64_t blocks = std::max<int64_t>(1, std::min({tiles * a.splits, launch_blocks(), int64_t(a.resident)}));
  if constexpr (DIR != S_WEIGHT)
    if (p.few) {
      if (a.chunk_rows <= 16) return s.launch(k_vocab_few<DT, DIR, KEEP, 1>, blocks, TileF<DT>::kThreads, a);
      return s.launch(k_vocab_few<DT, DIR, KEEP, 4>, blocks, TileF<DT>::kThreads, a);
    }
  if (z == Z_L) s.launch(k_vocab_product<TileL, DIR, KEEP>, blocks, TileL::kThreads, a);
  else if (z == Z_M) s.launch(k_vocab_product<TileM, DIR, KEEP>, blocks, TileM::kThreads, a);
  else if constexpr (DIR != S_WEIGHT) s.launch(k_vocab_product<TileS, DIR, KEEP>, blocks, TileS::kThreads, a);
}

template <int DT> RunResult run_typed(const Vocab& v, bool grad, const Plan& p, hipStream_t st) {
  char* ws = static_cast<char*>(v.workspace);
  Sequence s{st, {static_cast<hipEvent_t>(v.start_event), static_cast<hipEvent_t>(v.stop_event)}, 0};
  const int64_t P = int64_t(v.pieces.size());
  const bool each = v.reduction == R_NONE;
  const int64_t batches = (P + kPieceTab - 1) / kPieceTab, row_blocks = (p.Tpad + kRowWaves - 1) / kRowWaves;
  const bool sorted = p.Kp > kFewIds, pack_first = batches == 1 && v.T * p.Hp * p.planes <= kFewElements;
  const int64_t per_chunk = 2 + (grad ? 3 + sorted + p.hidden_part + (p.chunks == 1 && p.weight_splits > 1) : 0);
  s.left = batches + (v.top ? 1 : 0) + !pack_first + sorted + p.chunks * per_chunk + (grad ? p.chunks > 1 : !each);
  Piece* pieces = reinterpret_cast<Piece*>(ws + p.pieces);
  Counts* counts = reinterpret_cast<Counts*>(ws + p.counts);
  int32_t* rows = reinterpret_cast<int32_t*>(ws + p.rows);
  uint8_t* flags = reinterpret_cast<uint8_t*>(ws + p.flags);
  float2* teacher = reinterpret_cast<float2*>(ws + p.teacher);
  const Targets t{v.ids, v.logits, v.token_weights, v.ids_ld, v.logits_ld, v.ignore, p.V, v.top, v.logits_dtype, v.wide_ids, v.temperature};
  const PackArgs pa{v.hidden, v.ld, v.T, p.Tpad, int32_t(v.H), p.Hp, int32_t(P), pieces, rows, flags, counts, ws + p.hp,
                    reinterpret_cast<int32_t*>(ws + p.idt), p.Kp, p.lo, grad ? v.dh : nullptr, v.dh_ld, each ? v.loss : nullptr};
  if (v.top) s.launch(k_vocab_teacher, blocks_of(row_blocks), kRowWaves * 64, t, v.T, teacher, flags);
  int64_t first = 0, start = 0;
  for (int64_t i0 = 0; i0 < P; i0 += kPieceTab) {
    PrepareArgs pr{};
    pr.tab.at = int32_t(i0);
    pr.tab.count = int32_t(std::min<int64_t>(kPieceTab, P - i0));
    const int64_t before = start;
    for (int i = 0; i < pr.tab.count; ++i) {
      const VocabPiece& q = v.pieces[size_t(i0 + i)];
      pr.tab.p[i] = Piece{static_cast<const char*>(q.w), static_cast<char*>(q.dw), q.ld, q.dld, int32_t(q.rows), int32_t(start), int32_t(first), 0};
      first += q.rows;
      start += int64_t(up(size_t(q.rows), kUnit));
    }
    pr.pieces = pieces;
    pr.wp = p.packed ? ws + p.wp : nullptr;
    pr.scan = i0 == 0;
    pr.pack = pack_first;
    pr.mean = v.reduction == R_MEAN;
    pr.H = int32_t(v.H);
    pr.Hp = p.Hp;
    pr.T = v.T;
    pr.rows = rows;
    pr.flags = flags;
    pr.counts = counts;
    s.launch(k_vocab_prepare<DT>, p.packed ? blocks_of(1 + (start - before + kScanThreads / 64 - 1) / (kScanThreads / 64)) : 1, kScanThreads, pr, t, pa);
  }
  if (!pack_first) s.launch(k_vocab_pack<DT>, blocks_of(row_blocks), kRowWaves * 64, pa, t);
  if (sorted) {
    const int64_t row_tiles = p.Tpad / p.tile_rows;
    s.launch_lds(k_vocab_sort, blocks_of(row_tiles), kSortThreads, size_t(p.Vp / p.block + 1) * 4, pa.idt, p.Kp, p.tile_rows, p.block,
                 int(p.Vp / p.block), row_tiles, counts, reinterpret_cast<int32_t*>(ws + p.starts), reinterpret_cast<uint32_t*>(ws + p.entries));
  }
  Product a{};
  a.pieces = pieces;
  a.P = int32_t(P);
  a.H = int32_t(v.H);
  a.Hp = p.Hp;
  a.Vp = int32_t(p.Vp);
  a.planes = p.planes;
  a.kend = p.packed ? p.Hp : int32_t(v.H);  // (few rows' products go by H)
  a.hp = ws + p.hp;
  a.d = ws + p.d;
  a.scale = float(kLog2e / double(v.temperature));
  a.stats = reinterpret_cast<float2*>(ws + p.stats);
  a.ld_stats = p.Tc;
  a.idt = pa.idt;
  a.ld_idt = p.Kp;
  a.zt = reinterpret_cast<float*>(ws + p.zt);
  a.starts = reinterpret_cast<const int32_t*>(ws + p.starts);
  a.entries = reinterpret_cast<const uint32_t*>(ws + p.entries);
  a.entries_ld = p.tile_rows * p.Kp;
  a.rows = rows;
  a.dh = v.dh;
  a.dh_ld = v.dh_ld;
  Soft f{counts, rows, v.token_weights, a.stats, p.Tc, int32_t(p.Vp / p.block), 0, 0, v.reduction, p.planes, p.block, p.Vp,
         a.scale, reinterpret_cast<float2*>(ws + p.lse), reinterpret_cast<float*>(ws + p.coef), reinterpret_cast<float*>(ws + p.exps), ws + p.d, p.lo};
  const auto rows_of = [&](int64_t c) { return std::min(p.Tc, std::max<int64_t>(v.T - c * p.Tc, 0)); };
  const auto join_blocks = [&](int64_t n) { return blocks_of(int64_t(up(size_t(n), kUnit)) / kJoinRows); };
  Ends ends{teacher, pa.idt, p.Kp, a.zt, reinterpret_cast<float*>(ws + p.row_loss), each ? v.loss : nullptr, nullptr};
  float* dh_part = reinterpret_cast<float*>(ws + p.part);
  float* dw_part = dh_part;
  if (p.chunks > 1 && p.hidden_part) dw_part += size_t(p.hidden_splits) * size_t(p.Tc) * size_t(p.Hp);
  for (int64_t c = 0; c < p.chunks; ++c) {
    a.chunk = f.chunk = int32_t(c * p.Tc);
    a.chunk_rows = f.chunk_rows = int32_t(rows_of(c));
    const int64_t n = a.chunk_rows, npad = int64_t(up(size_t(n), kUnit));
    const auto tile = [&](Size z) {
      a.bn = int32_t(z == Z_L ? 256 : z == Z_M ? 128 : 64);
      a.resident = z == Z_L ? kUnits : 2 * kUnits;
    };
    tile(p.logits);
    a.mtiles = int32_t(p.Vp / p.block);
    a.splits = 1;
    a.part = f.exps;
    const int64_t tiles = tiles_of(p.logits, p.Vp, n);
    if (grad) launch_product<DT, S_LOGITS, DT>(s, p, p.logits, tiles, a);
    else launch_product<DT, S_LOGITS, 0>(s, p, p.logits, tiles, a);
    s.launch(k_vocab_join, join_blocks(n), kJoinThreads, f, ends, t);
    const bool total = !each && c + 1 == p.chunks;
    ends.total = total ? v.loss : nullptr;
    if (!grad) {
      if (total) s.launch(k_vocab_total, 1, kNormThreads, f, ends);
      continue;
    }
    s.launch(k_vocab_normalize<DT>, blocks_of(npad / kNormRows * ((p.Vp + kNormCols - 1) / kNormCols) + total), kNormThreads, f, ends, t);
    if (sorted) s.launch(k_vocab_own<DT>, blocks_of((n * ((p.Kp + 63) / 64) + 3) / 4), 256, f, ends, t);
    const auto mtiles = [&](Size z) { return int32_t(tiles_of(z, v.H, 1)); };
    tile(p.hidden);
    a.mtiles = mtiles(p.hidden);
    a.splits = p.hidden_splits;
    a.part = p.hidden_part ? dh_part : nullptr;
    a.lo = p.lo;
    a.part_stride = p.Tc * p.Hp;
    a.accumulate = 0;
    launch_product<DT, S_HIDDEN, DT>(s, p, p.hidden, tiles_of(p.hidden, v.H, p.lo ? 2 * p.lo : n), a);
    if (p.few) a.lo = 0;  // (its products are of both terms)
    if (a.part) s.launch(k_vocab_sum<S_HIDDEN, DT>, blocks_of((n * p.Hp / 4 + 255) / 256), 256, a);
    tile(p.weight);
    a.mtiles = mtiles(p.weight);
    a.splits = p.weight_splits;
    a.part = a.splits > 1 || p.chunks > 1 ? dw_part : nullptr;
    a.part_stride = p.Vp * p.Hp;
    a.accumulate = c > 0;
    a.lo = p.lo;
    launch_product<DT, S_WEIGHT, DT>(s, p, p.weight, tiles_of(p.weight, v.H, p.Vp), a);
    if (a.part && c + 1 == p.chunks) s.launch(k_vocab_sum<S_WEIGHT, DT>, blocks_of((p.Vp * p.Hp / 4 + 255) / 256), 256, a);
  }
  return s.done("launching the vocabulary kernels");
}

}  // namespace

size_t vocab_workspace(const Vocab& v, bool grad) { return plan_of(v, grad).bytes; }

RunResult run_vocab(const Vocab& v, bool grad, void* stream) {
  const Plan p = plan_of(v, grad);
  if (v.workspace_bytes < p.bytes) {
    RunResult r;
    r.status = 3;
    r.message = "workspace too small: need " + std::to_string(p.bytes) + " bytes";
    return r;
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return v.dtype == D_FP32 ? run_typed<D_FP32>(v, grad, p, st) : run_typed<D_BF16>(v, grad, p, st);
}

}  // namespace ar
