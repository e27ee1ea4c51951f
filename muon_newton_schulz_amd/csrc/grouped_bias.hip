// The gradient of a layer's bias, for rows sorted by expert: dZ = dY act'(Z) and db_e = the sum of
// dZ's rows of expert e.
//
// Bound by HBM: dY and Z are read once and dZ is written once, with no reuse (16384 rows x 8192, bfloat16, gelu,
// 805 MB: 146 + 9 us, 5.5 TB/s; with accesses that stay in the caches 173, so operands beyond the last-level
// cache take non-temporal ones). A block takes a chunk of
// `chunk` rows of one expert x 256 columns, eight columns a thread (16 bytes of bfloat16), eight rows
// side by side; its float32 column sums go to the workspace, one row of 256 a chunk, and are added by a
// second launch in chunk order, so equal calls give equal bits. An expert of at most one chunk needs
// no second launch; nor does a call of at most `chunk` rows.
#include "activation.h"
#include "grouped_walk.h"
#include "row_vectors.h"

namespace mns {
namespace {

constexpr int kCols = 256;                    // columns of a block
constexpr int kRowsAtOnce = 8;                // rows a block reads side by side

struct BiasArgs : GroupedArgs {               // A: dY (lda), C: dZ (ldc), B: Z (ldb), D: unused
  void* db;                                   // groups x N
  int act;
  int chunk;                                  // rows, a multiple of kRowsAtOnce
};

template <typename T, typename TO, bool STREAM>
__global__ __launch_bounds__(256) void k_bias_grad(BiasArgs p) {
  const int tid = threadIdx.x, cg = tid & 31, rg = tid >> 5;
  Place at;
  const int lin = block_place();
  if (!find_place(p, p.chunk, p.tiles_n, p.fill_rest,
                  walk_start(p, p.chunk, p.tiles_n, p.fill_rest, 1), lin, at, 1))
    return;
  const int part = at.inside / p.tiles_n, n = at.inside % p.tiles_n * kCols + 8 * cg;
  const int left = p.N - n;
  const int64_t r0 = at.lo + (int64_t)part * p.chunk;
  const int rows = at.hi - r0 < p.chunk ? (int)(at.hi - r0) : p.chunk;
  const T* dY = static_cast<const T*>(p.A) + r0 * p.lda + n;
  const T* Z = static_cast<const T*>(p.B) + r0 * p.ldb + n;
  T* dZ = static_cast<T*>(p.C) + r0 * p.ldc + n;
  const T* dy_end = rows_end(static_cast<const T*>(p.A), p, p.lda, p.N);
  const T* z_end = rows_end(static_cast<const T*>(p.B), p, p.ldb, p.N);
  if (at.expert < 0) {                        // rows of no expert
    Eight<T> zero;
    const float none[8] = {};
    zero.set(none);
    for (int m = rg; m < rows; m += kRowsAtOnce) zero.store(dZ + m * p.ldc, left);
    return;
  }
  float sum[8] = {};
  constexpr int AHEAD = 4;                    // rows a thread loads before it uses the first
  for (int m = rg; m < rows; m += AHEAD * kRowsAtOnce) {
    Eight<T> g[AHEAD], z[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int r = m + q * kRowsAtOnce, have = r < rows ? left : 0;
      g[q].template load<STREAM>(dY + r * p.lda, have, dy_end);
      z[q].template load<STREAM>(Z + r * p.ldb, p.act ? have : 0, z_end);
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int r = m + q * kRowsAtOnce;
      if (r >= rows) continue;
      float v[8], x[8];
      g[q].get(v);
      z[q].get(x);
      times_slope<sizeof(T) == 4>(p.act, v, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[e];
      if (p.C) {
        Eight<T> out;
        out.set(v);
        out.template store<STREAM>(dZ + r * p.ldc, left);
      }
    }
  }
  __shared__ float part_sum[kRowsAtOnce][kCols];
#pragma unroll
  for (int e = 0; e < 8; ++e) part_sum[rg][8 * cg + e] = sum[e];
  __syncthreads();
  float total = 0.f;
#pragma unroll
  for (int r = 0; r < kRowsAtOnce; ++r) total += part_sum[r][tid];
  const int col = at.inside % p.tiles_n * kCols + tid;
  if (at.hi - at.lo <= p.chunk) {
    if (col < p.N) static_cast<TO*>(p.db)[(int64_t)at.expert * p.N + col] = (TO)total;
  } else {
    p.partial[(int64_t)lin * kCols + tid] = total;
  }
}

// One block per expert and 256 columns, which only experts of several chunks keep: it adds the chunks' sums,
// four quarters of them side by side (each in order), then the quarters in order. Latency of dependent loads
// from L2: 9 us for 32 experts of 8192, 27 with one block of 256 threads that walks all chunks.
template <typename TO>
__global__ __launch_bounds__(1024) void k_bias_join(BiasArgs p) {
  const int expert = block_place() / p.tiles_n, column_tile = block_place() % p.tiles_n;
  if (expert >= p.groups) return;
  int lo, hi;
  expert_rows(p, expert, lo, hi);
  if (hi - lo <= p.chunk) return;
  // its first chunk's place in the list of tiles: behind those of the entries before it
  Walk w;
  const int entry = expert + p.fill_rest;
  int64_t first = 0;
  for (int g0 = 0; g0 <= entry; g0 += 64) {
    walk_batch(p, p.chunk, p.tiles_n, p.fill_rest, g0, w, 1);
    const int at = entry - g0 < 64 ? entry - g0 : 64;
    if (at > 0) first += (unsigned)__builtin_amdgcn_readlane(w.incl, at - 1);
  }
  int64_t chunks = (hi - lo + p.chunk - 1) / p.chunk;
  const int64_t listed = (p.most_tiles - first) / p.tiles_n;      // fewer only where offsets overlap
  if (chunks > listed) chunks = listed;
  const int tid = threadIdx.x & 255, quarter = threadIdx.x >> 8;
  const int c0 = (int)(chunks * quarter / 4), c1 = (int)(chunks * (quarter + 1) / 4);
  float total = 0.f;
#pragma unroll 8
  for (int c = c0; c < c1; ++c)
    total += p.partial[(first + (int64_t)c * p.tiles_n + column_tile) * kCols + tid];
  __shared__ float part_sum[4][kCols];
  part_sum[quarter][tid] = total;
  __syncthreads();
  const int col = column_tile * kCols + tid;
  if (quarter == 0 && col < p.N)
    static_cast<TO*>(p.db)[(int64_t)expert * p.N + col] =
        (TO)(part_sum[0][tid] + part_sum[1][tid] + part_sum[2][tid] + part_sum[3][tid]);
}

template <bool STREAM>
hipError_t launch_bias(const BiasArgs& a, Store store, bool out32, dim3 grid, hipStream_t s) {
  if (store == Store::F32)
    hipLaunchKernelGGL((k_bias_grad<float, float, STREAM>), grid, dim3(256), 0, s, a);
  else if (out32)
    hipLaunchKernelGGL((k_bias_grad<__bf16, float, STREAM>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_bias_grad<__bf16, __bf16, STREAM>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

// Rows of a chunk: up to 128 rows one, and one launch; beyond 32 to 128, as many as leave 1024 blocks (us
// without / with gelu: 2048 rows x 1024, chunks of 32 8.1 / 10.2, of 64 8.9 / 12.6, of 128 11.6 / 17.7;
// 16384 x 1024: 14.7 / 28.4, 11.6 / 24.6, 13.4 / 28.3; 16384 x 8192: 78 / 150, 57 / 146, 52 / 151, of 256
// 51 / 163); more only where there would be more than 512 chunks of a column to join.
int chunk_rows(int64_t total_rows, int64_t n) {
  const int64_t columns = (n + kCols - 1) / kCols;
  int64_t c = total_rows <= 128 ? 128 : 32;
  while (c < 128 && total_rows * columns > 1024 * c) c *= 2;
  while (total_rows > 512 * c) c *= 2;
  return (int)c;
}

}  // namespace

int64_t bias_grad_blocks(int64_t groups, int64_t total_rows, int64_t n) {
  const int64_t chunk = chunk_rows(total_rows, n);
  return ((total_rows + chunk - 1) / chunk + groups + 2) * ((n + kCols - 1) / kCols);
}

size_t bias_grad_workspace(int64_t groups, int64_t total_rows, int64_t n) {
  if (total_rows <= chunk_rows(total_rows, n)) return 0;
  return (size_t)bias_grad_blocks(groups, total_rows, n) * kCols * sizeof(float);
}

hipError_t bias_grad(const BiasGradDesc& d, hipStream_t s) {
  BiasArgs a = {};
  a.A = d.dY; a.lda = d.lddy;
  a.B = d.Z; a.ldb = d.ldz;
  a.C = d.dZ; a.ldc = d.lddz;
  a.offsets = d.offsets;
  a.total_rows = (int)d.total_rows;
  a.groups = (int)d.groups;
  a.N = (int)d.n;
  a.tiles_n = (int)((d.n + kCols - 1) / kCols);
  const int64_t blocks = bias_grad_blocks(d.groups, d.total_rows, d.n);
  a.most_tiles = (int)blocks;
  a.fill_rest = d.dZ && d.fill_rest ? 1 : 0;
  a.partial = d.workspace;
  a.db = d.db;
  a.act = d.act;
  a.chunk = chunk_rows(d.total_rows, d.n);
  const dim3 grid = grid_of(blocks);
  const bool out32 = d.out_store == Store::F32;
  const double bytes = (double)d.total_rows * d.n * (d.store == Store::F32 ? 4 : 2) *
                       (1 + (d.Z ? 1 : 0) + (d.dZ ? 1 : 0));
  const hipError_t e = bytes > kStreamBytes ? launch_bias<true>(a, d.store, out32, grid, s)
                                            : launch_bias<false>(a, d.store, out32, grid, s);
  if (e != hipSuccess || d.total_rows <= a.chunk) return e;
  const dim3 joins = grid_of(d.groups * a.tiles_n);
  if (out32) hipLaunchKernelGGL(k_bias_join<float>, joins, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL(k_bias_join<__bf16>, joins, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace mns
