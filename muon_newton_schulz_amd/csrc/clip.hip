// The global norm over many gradients, and their scaling by min(1, max_norm / (norm + eps)).
//
// Both passes are bound by HBM: the norm reads every gradient once, the scaling reads and writes it once.
// Every tensor is cut into pieces of 16 KB, which a grid of at most kNormBlocks (kScaleBlocks) blocks
// deals out in turn; the tensors' pointers and first pieces travel as kernel arguments, kClipPack tensors a launch,
// so nothing is uploaded. Squares are formed and added in float64 (as everywhere in this library: no
// underflow or overflow for any float32 gradient), a partial sum per block; every block of the scaling
// adds all partial sums itself, in the same order, instead of waiting for a launch in between that
// would do nothing else. The scaling walks the pieces backwards: those read last are still in the caches.
#include "mns_internal.h"
#include "row_vectors.h"

namespace mns {
namespace {

constexpr int kThreads = 256;
constexpr int kPieceBytes = 16384;
constexpr int kNormBlocks = 2048, kScaleBlocks = 2048;

struct Table {
  struct Entry {
    const void* in;
    void* out;
    int64_t numel;
    int64_t first;              // piece
  } t[kClipPack];
  int count, f32_from;          // tensors from f32_from on are float32
  int64_t pieces;
};

// The tensor of piece i: the last one whose first piece is not behind it (uniform: scalar registers).
__device__ __forceinline__ int tensor_of(const Table& a, int64_t i) {
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.t[mid].first <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The n elements of a piece (more: of a whole one), zeros behind them.
template <typename T>
__device__ __forceinline__ void load_piece(const T* p, int64_t n, u32x4* v) {
  constexpr int VEC = 16 / sizeof(T), PER = kPieceBytes / 16 / kThreads;
  const bool whole = n >= kPieceBytes / (int)sizeof(T);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int at = (q * kThreads + threadIdx.x) * VEC;
    v[q] = load_chunk(p + at, whole ? VEC : (int)n - at);
  }
}

template <typename T>
__device__ __forceinline__ double piece_squares(const T* p, int64_t n) {
  constexpr int VEC = 16 / sizeof(T), PER = kPieceBytes / 16 / kThreads;
  u32x4 v[PER];
  load_piece<T>(p, n, v);
  double s[PER] = {};
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    T e[VEC];
    __builtin_memcpy(e, &v[q], 16);
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[q] = fma((double)(float)e[i], (double)(float)e[i], s[q]);
  }
  double all = 0.;
#pragma unroll
  for (int q = 0; q < PER; ++q) all += s[q];
  return all;
}

// (result in every thread of the block)
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double waves[kThreads / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
  __syncthreads();
  double all = 0.;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) all += waves[w];
  return all;
}

__global__ __launch_bounds__(kThreads) void k_grad_squares(Table a, double* partial) {
  double sum = 0.;
  for (int64_t i = blockIdx.x; i < a.pieces; i += gridDim.x) {
    const int t = tensor_of(a, i);
    const int64_t k = i - a.t[t].first;
    if (t >= a.f32_from) {
      const int64_t at = k * (kPieceBytes / 4);
      sum += piece_squares(static_cast<const float*>(a.t[t].in) + at, a.t[t].numel - at);
    } else {
      const int64_t at = k * (kPieceBytes / 2);
      sum += piece_squares(static_cast<const __bf16*>(a.t[t].in) + at, a.t[t].numel - at);
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* p, T* out, int64_t n, float factor) {
  constexpr int VEC = 16 / sizeof(T), PER = kPieceBytes / 16 / kThreads;
  u32x4 v[PER];
  load_piece<T>(p, n, v);
  const bool whole = n >= kPieceBytes / (int)sizeof(T);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int at = (q * kThreads + threadIdx.x) * VEC;
    T e[VEC];
    __builtin_memcpy(e, &v[q], 16);
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = (T)((float)e[i] * factor);
    if (whole || at + VEC <= (int)n) {
      __builtin_memcpy(out + at, e, 16);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (at + i < (int)n) out[at + i] = e[i];
    }
  }
}

// norm: written by block 0 of the first launch (null in the others).
__global__ __launch_bounds__(kThreads) void k_grad_scale(Table a, const double* partial, int partials,
                                                         float max_norm, float eps, float* norm) {
  double sum = 0.;
  for (int i = threadIdx.x; i < partials; i += kThreads) sum += partial[i];
  const double total = sqrt(block_sum(sum));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
  const double floor = total + (double)eps, ratio = (double)max_norm / floor;
  const float factor = ratio >= 1. || floor == 0. ? 1.f : (float)ratio;       // a NaN stays one
  for (int64_t b = blockIdx.x; b < a.pieces; b += gridDim.x) {
    const int64_t i = a.pieces - 1 - b;
    const int t = tensor_of(a, i);
    if (factor == 1.f && a.t[t].in == a.t[t].out) continue;
    const int64_t k = i - a.t[t].first;
    if (t >= a.f32_from) {
      const int64_t at = k * (kPieceBytes / 4);
      scale_piece(static_cast<const float*>(a.t[t].in) + at, static_cast<float*>(a.t[t].out) + at,
                  a.t[t].numel - at, factor);
    } else {
      const int64_t at = k * (kPieceBytes / 2);
      scale_piece(static_cast<const __bf16*>(a.t[t].in) + at, static_cast<__bf16*>(a.t[t].out) + at,
                  a.t[t].numel - at, factor);
    }
  }
}

// Tensors [first, first + kClipPack) of the list, bfloat16 ones before float32 ones.
void fill_table(Table& a, const ClipTensor* list, int count) {
  a.count = 0;
  a.pieces = 0;
  for (int pass = 0; pass < 2; ++pass) {
    const Store st = pass == 0 ? Store::BF16 : Store::F32;
    if (pass == 1) a.f32_from = a.count;
    const int64_t per = kPieceBytes / (st == Store::F32 ? 4 : 2);
    for (int i = 0; i < count; ++i) {
      if (list[i].store != st || list[i].numel == 0) continue;
      a.t[a.count++] = {list[i].in, list[i].out, list[i].numel, a.pieces};
      a.pieces += (list[i].numel + per - 1) / per;
    }
  }
}

int grid_of(const Table& a, int most) { return (int)(a.pieces < most ? a.pieces : most); }

}  // namespace

size_t clip_workspace(int count) {
  return (size_t)((count + kClipPack - 1) / kClipPack) * kNormBlocks * sizeof(double);
}

hipError_t clip_grads(const ClipTensor* list, int count, bool scale, float max_norm, float eps,
                      float* norm, double* partial, hipStream_t s) {
  int partials = 0;
  Table a;
  for (int i = 0; i < count; i += kClipPack) {
    fill_table(a, list + i, count - i < kClipPack ? count - i : kClipPack);
    if (a.pieces == 0) continue;
    const int grid = grid_of(a, kNormBlocks);
    hipLaunchKernelGGL(k_grad_squares, dim3((unsigned)grid), dim3(kThreads), 0, s, a, partial + partials);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    partials += grid;
  }
  // The first launch also writes the norm; without scaling, or without elements, it does only that.
  for (int i = 0; i < count; i += kClipPack) {
    fill_table(a, list + i, scale ? (count - i < kClipPack ? count - i : kClipPack) : 0);
    if (a.pieces == 0 && i > 0) continue;
    const int grid = a.pieces == 0 ? 1 : grid_of(a, kScaleBlocks);
    hipLaunchKernelGGL(k_grad_scale, dim3((unsigned)grid), dim3(kThreads), 0, s, a, partial, partials,
                       max_norm, eps, i == 0 ? norm : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !scale) return e;
  }
  return hipSuccess;
}

}  // namespace mns
