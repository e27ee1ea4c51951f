// The global norm over many gradients, and their scaling by min(1, max_norm / (norm + eps)).
//
// Both passes are bound by HBM: the norm reads every gradient once, the scaling reads and writes it once.
// Every tensor is cut into pieces of 16 KB; the tensors' pointers and first pieces travel as kernel
// arguments, kClipPack tensors a launch, so nothing is uploaded. Squares are formed and added in float64
// (as everywhere in this library: no underflow or overflow for any float32 gradient), a partial sum per
// block of at most kNormBlocks, added in the same order by everyone who needs the norm.
//
// Few pieces (kFewPieces): every block of the scaling adds the partial sums itself, which takes less than a
// launch in between (four tensors, us, and with that launch: 64 KB 5.0, 6.3; 6.5 MB 6.0, 7.1; 24 MB 7.8, 8.4;
// 32 MB 10.0, 9.9). More: a launch of one block adds them, and each block of the scaling takes one piece
// (1.5 GB, out of place: 490 us; blocks that go from piece to piece 8 to 11 % longer). Lists beyond the 256 MB
// last-level cache are read and written with non-temporal accesses (1.5 GB: the norm 224 us, the scaling 490; with
// ordinary ones 15 and 10 % longer); smaller ones stay in the caches for the step that follows. Walking the
// pieces backwards, so that those read last are found in the caches, gained nothing.
#include "mns_internal.h"
#include "row_vectors.h"

namespace mns {
namespace {

constexpr int kThreads = 256;
constexpr int kPieceBytes = 16384;
constexpr int kNormBlocks = 2048, kFewPieces = 2048;

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

// The tensor that holds the pieces a block comes to, one after the other: looked up in the arguments only
// when a piece lies outside the current one (uniform: scalar registers).
struct Cursor {
  const void* in;
  void* out;
  int64_t numel, first, end;    // pieces [first, end)
  bool f32;
  __device__ __forceinline__ void to(const Table& a, int64_t i) {
    int lo = 0, hi = a.count;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.t[mid].first <= i) lo = mid;
      else hi = mid;
    }
    in = a.t[lo].in;
    out = a.t[lo].out;
    numel = a.t[lo].numel;
    first = a.t[lo].first;
    end = lo + 1 < a.count ? a.t[lo + 1].first : a.pieces;
    f32 = lo >= a.f32_from;
  }
};

// The n elements of a piece (more: of a whole one), zeros behind them.
template <typename T, bool STREAM>
__device__ __forceinline__ void load_piece(const T* p, int64_t n, u32x4* v) {
  constexpr int VEC = 16 / sizeof(T), PER = kPieceBytes / 16 / kThreads;
  if (n >= kPieceBytes / (int)sizeof(T)) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const T* at = p + (q * kThreads + threadIdx.x) * VEC;
      if (STREAM) v[q] = load_streaming(at);
      else __builtin_memcpy(&v[q], at, 16);
    }
  } else {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int at = (q * kThreads + threadIdx.x) * VEC;
      v[q] = load_chunk(p + at, (int)n - at);
    }
  }
}

template <typename T, bool STREAM>
__device__ __forceinline__ double piece_squares(const T* p, int64_t n) {
  constexpr int VEC = 16 / sizeof(T), PER = kPieceBytes / 16 / kThreads;
  u32x4 v[PER];
  load_piece<T, STREAM>(p, n, v);
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

template <bool STREAM>
__global__ __launch_bounds__(kThreads) void k_grad_squares(Table a, double* partial) {
  double sum = 0.;
  Cursor c;
  c.end = 0;
  for (int64_t i = blockIdx.x; i < a.pieces; i += gridDim.x) {
    if (i >= c.end) c.to(a, i);
    const int64_t at = (i - c.first) * (kPieceBytes / (c.f32 ? 4 : 2));
    if (c.f32) sum += piece_squares<float, STREAM>(static_cast<const float*>(c.in) + at, c.numel - at);
    else sum += piece_squares<__bf16, STREAM>(static_cast<const __bf16*>(c.in) + at, c.numel - at);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <typename T, bool STREAM>
__device__ __forceinline__ void scale_piece(const T* p, T* out, int64_t n, float factor) {
  constexpr int VEC = 16 / sizeof(T), PER = kPieceBytes / 16 / kThreads;
  u32x4 v[PER];
  load_piece<T, STREAM>(p, n, v);
  const bool whole = n >= kPieceBytes / (int)sizeof(T);
#pragma unroll
  for (int q = 0; q < PER; ++q) {
    const int at = (q * kThreads + threadIdx.x) * VEC;
    T e[VEC];
    __builtin_memcpy(e, &v[q], 16);
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = (T)((float)e[i] * factor);
    if (STREAM && whole) {
      store_streaming(out + at, e);
    } else if (whole || at + VEC <= (int)n) {
      __builtin_memcpy(out + at, e, 16);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (at + i < (int)n) out[at + i] = e[i];
    }
  }
}

// The norm and the factor from the partial sums (in every thread of the block).
__device__ __forceinline__ float clip_factor(const double* partial, int partials, float max_norm,
                                             float eps, double& total) {
  double sum = 0.;
#pragma unroll 4
  for (int i = threadIdx.x; i < partials; i += kThreads) sum += partial[i];
  total = sqrt(block_sum(sum));
  const double floor = total + (double)eps;
  return (double)max_norm >= floor ? 1.f : (float)((double)max_norm / floor);   // a NaN stays one
}

__global__ __launch_bounds__(kThreads) void k_grad_norm(const double* partial, int partials,
                                                        float max_norm, float eps, float* norm,
                                                        float* factor) {
  double total;
  const float f = clip_factor(partial, partials, max_norm, eps, total);
  if (threadIdx.x == 0) {
    *norm = (float)total;
    *factor = f;
  }
}

// One piece a block. factor null: from the partial sums, and block 0 writes the norm.
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void k_grad_scale(Table a, const double* partial, int partials,
                                                         float max_norm, float eps, float* norm,
                                                         const float* factor) {
  float f;
  if (factor) {
    f = *factor;
  } else {
    double total;
    f = clip_factor(partial, partials, max_norm, eps, total);
    if (block_place() == 0 && threadIdx.x == 0) *norm = (float)total;
  }
  const int64_t piece = block_place();
  if (piece >= a.pieces) return;
  Cursor c;
  c.to(a, piece);
  if (f == 1.f && c.in == c.out) return;
  const int64_t at = (piece - c.first) * (kPieceBytes / (c.f32 ? 4 : 2));
  if (c.f32)
    scale_piece<float, STREAM>(static_cast<const float*>(c.in) + at, static_cast<float*>(c.out) + at,
                               c.numel - at, f);
  else
    scale_piece<__bf16, STREAM>(static_cast<const __bf16*>(c.in) + at,
                                static_cast<__bf16*>(c.out) + at, c.numel - at, f);
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

}  // namespace

// The partial sums, and the factor behind them.
size_t clip_workspace(int count) {
  return (size_t)((count + kClipPack - 1) / kClipPack) * kNormBlocks * sizeof(double) + 256;
}

hipError_t clip_grads(const ClipTensor* list, int count, bool scale, float max_norm, float eps,
                      float* norm, double* partial, hipStream_t s) {
  double bytes = 0;
  for (int i = 0; i < count; ++i) bytes += (double)list[i].numel * (list[i].store == Store::F32 ? 4 : 2);
  const bool stream = bytes > kStreamBytes;
  float* factor = reinterpret_cast<float*>(partial + clip_workspace(count) / sizeof(double) - 32);
  const dim3 block(kThreads);
  int partials = 0;
  int64_t pieces = 0;
  Table a;
  hipError_t e;
  for (int i = 0; i < count; i += kClipPack) {
    fill_table(a, list + i, count - i < kClipPack ? count - i : kClipPack);
    if (a.pieces == 0) continue;
    const int grid = (int)(a.pieces < kNormBlocks ? a.pieces : kNormBlocks);
    if (stream) hipLaunchKernelGGL(k_grad_squares<true>, dim3((unsigned)grid), block, 0, s, a, partial + partials);
    else hipLaunchKernelGGL(k_grad_squares<false>, dim3((unsigned)grid), block, 0, s, a, partial + partials);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    partials += grid;
    pieces += a.pieces;
  }
  const bool few = scale && count <= kClipPack && pieces > 0 && pieces <= kFewPieces;
  if (!few) {
    hipLaunchKernelGGL(k_grad_norm, dim3(1), block, 0, s, partial, partials, max_norm, eps, norm, factor);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  for (int i = 0; scale && i < count; i += kClipPack) {
    if (count > kClipPack) fill_table(a, list + i, count - i < kClipPack ? count - i : kClipPack);
    if (a.pieces == 0) continue;
    const dim3 grid = grid_of(a.pieces);
    const float* given = few ? nullptr : factor;
    if (stream) hipLaunchKernelGGL(k_grad_scale<true>, grid, block, 0, s, a, partial, partials, max_norm, eps, norm, given);
    else hipLaunchKernelGGL(k_grad_scale<false>, grid, block, 0, s, a, partial, partials, max_norm, eps, norm, given);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mns
