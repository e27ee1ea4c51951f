// Memory-bound kernels of the Newton-Schulz gradient (ns_orthogonalize_backward); its products
// run on the GEMM of gemm.hip.
//
// O = NS_T(X / ||X||_F) acts on the singular values alone, so its derivative at X_0 = X / ||X||
// is symmetric as a linear map: in the singular basis it scales the symmetric part of a direction
// by (f_i - f_j) / (s_i - s_j), the skew part by (f_i + f_j) / (s_i + s_j) and the rectangular
// part by f_i / s_i. The gradient J^T dO therefore equals the derivative J dO in the direction
// dO, which is carried along the iteration instead of walking back through stored iterates:
//
//   A = X X^T,  S = E X^T + X E^T,  P = a I + b A + c A^2,  Q = b S + c (A S + S A),
//   E <- P E + Q X,  X <- P X              (E_0 = dO)
//
// and dX = (E_T - X_0 <X_0, E_T>) / ||X||, the normalisation's (symmetric) derivative.
#include "lds_dma.h"
#include "mns_internal.h"

namespace mns {
namespace {

constexpr int kT = 64;      // tile of the transposing kernels
constexpr int kThreads = 256;

__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ void narrow(double v, float* o) { *o = (float)v; }
// float64 -> bfloat16 through float32, to odd: the float32 value is forced to the odd neighbour
// when inexact, so that the second rounding (to nearest even) sees which side it came from and
// the result is the one rounding of v.
__device__ __forceinline__ void narrow(double v, uint16_t* o) {
  float f = (float)v;
  uint32_t u = __float_as_uint(f);
  if (f != f) {
    *o = 0x7FC0;
    return;
  }
  const double back = (double)f;
  if (back != v && isfinite(f)) {
    if (fabs(back) > fabs(v)) --u;     // truncate towards zero ...
    u |= 1u;                           // ... and make it odd
  }
  u += 0x7FFFu + ((u >> 16) & 1u);
  *o = (uint16_t)(u >> 16);
}

// Eight consecutive elements, 16-byte (or twice 16-byte) loads and stores; the addresses are aligned
// where the row length is a multiple of 8.
__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const _Float16* p, float* v) {
  typedef _Float16 half8 __attribute__((ext_vector_type(8)));
  const half8 h = *reinterpret_cast<const half8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const T* v) {
  typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
  constexpr int N = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 8; i += N) {
    vec x;
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = v[i + e];
    *reinterpret_cast<vec*>(p + i) = x;
  }
}

// scale[4 b ..]: S / ||X||, 1 / ||X||, e0 / ||dO||, ||dO|| of matrix b (zeros for a zero norm),
// from nblk partial sums of squares of X and, behind them, of dO. exact: the first and third rounded
// down to powers of two, so that in float16 a bfloat16 element keeps every bit if its scaled magnitude is
// at least 2^-17 (below, float16's smallest step of 2^-24 cuts bits off); k_nsb_square makes up for X's in
// the first iteration, and the fourth is e0 / (third).
__global__ __launch_bounds__(kThreads) void k_nsb_scales(const double* px, const double* pg,
                                                         int nblk, double S, double e0,
                                                         bool exact, double* scale) {
  __shared__ double red[2][kThreads];
  const int b = blockIdx.x;
  double sx = 0.0, sg = 0.0;
  for (int i = threadIdx.x; i < nblk; i += kThreads) {
    sx += px[(int64_t)b * nblk + i];
    sg += pg[(int64_t)b * nblk + i];
  }
  red[0][threadIdx.x] = sx;
  red[1][threadIdx.x] = sg;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) {
      red[0][threadIdx.x] += red[0][threadIdx.x + o];
      red[1][threadIdx.x] += red[1][threadIdx.x + o];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double nx = sqrt(red[0][0]), ng = sqrt(red[1][0]);
    const double sx = nx == 0.0 ? 0.0 : S / nx, sg = ng == 0.0 ? 0.0 : e0 / ng;
    const bool px2 = exact && nx > 0.0 && nx < 1e300, pg2 = exact && ng > 0.0 && ng < 1e300;
    scale[4 * b] = px2 ? ldexp(1.0, ilogb(sx)) : sx;
    scale[4 * b + 1] = nx == 0.0 ? 0.0 : 1.0 / nx;
    scale[4 * b + 2] = pg2 ? ldexp(1.0, ilogb(sg)) : sg;
    scale[4 * b + 3] = pg2 ? e0 / ldexp(1.0, ilogb(sg)) : ng;
  }
}

// E_0 and X_0 (scaled, zero padded) from dO and X, in either layout or both. Destination
// elements: straight[b * stride + which * offset + r * ld + c] for source element (r, c), and
// likewise transposed[... + c * ld + r]; which = 0 for dO (E), 1 for X.
struct LoadDst {
  void* p;
  int64_t ld, stride, offset;
};
template <typename TX, typename TO>
__global__ __launch_bounds__(kThreads) void k_nsb_load(const TX* X, const TX* G, int64_t rows,
                                                       int64_t cols, int64_t elems,
                                                       const double* scale, LoadDst st,
                                                       LoadDst tr) {
  __shared__ TO tile[kT][kT + 2];
  const int b = blockIdx.z >> 1, which = blockIdx.z & 1;
  const int64_t r0 = (int64_t)blockIdx.y * kT, c0 = (int64_t)blockIdx.x * kT;
  const TX* src = (which ? X : G) + b * elems;
  const double sc = scale[4 * b + (which ? 0 : 2)];
  const int lx = threadIdx.x % kT, ly = threadIdx.x / kT;
#pragma unroll
  for (int i = 0; i < kT; i += kThreads / kT) {
    const int64_t r = r0 + ly + i, c = c0 + lx;
    double v = 0.0;
    if (r < rows && c < cols) v = (double)widen(src[r * cols + c]) * sc;
    const TO o = (TO)(float)v;
    if (st.p) static_cast<TO*>(st.p)[b * st.stride + which * st.offset + r * st.ld + c] = o;
    tile[ly + i][lx] = o;
  }
  if (!tr.p) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kT; i += kThreads / kT) {
    const int64_t r = r0 + lx, c = c0 + ly + i;
    static_cast<TO*>(tr.p)[b * tr.stride + which * tr.offset + c * tr.ld + r] = tile[lx][ly + i];
  }
}

// The straight layout alone (a wide matrix whose products read the iterate as it is stored): rows of
// 8-element vectors, bound by its bytes (4096 x 16384: 81 us, 6.6 TB/s). blockIdx.y: padded row;
// blockIdx.z as above.
template <typename TX, typename TO>
__global__ __launch_bounds__(kThreads) void k_nsb_load_rows(const TX* X, const TX* G, int64_t rows,
                                                            int64_t cols, int64_t cols_p,
                                                            int64_t elems, const double* scale,
                                                            LoadDst st) {
  const int b = blockIdx.z >> 1, which = blockIdx.z & 1;
  const int64_t r = blockIdx.y;
  const TX* src = (which ? X : G) + b * elems + r * cols;
  TO* dst = static_cast<TO*>(st.p) + b * st.stride + which * st.offset + r * st.ld;
  const double sc = scale[4 * b + (which ? 0 : 2)];
  const bool vec = cols % 8 == 0;
  // four vectors of a thread in flight together
  const int64_t c0 = ((int64_t)blockIdx.x * 4 * kThreads + threadIdx.x) * 8;
  float v[4][8];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t c = c0 + u * kThreads * 8;
    if (r < rows && c < cols && vec) {
      load8(src + c, v[u]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] = r < rows && c + e < cols ? widen(src[c + e]) : 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t c = c0 + u * kThreads * 8;
    if (c >= cols_p) break;
    TO o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (TO)(float)((double)v[u][e] * sc);
    store8(dst + c, o);
  }
}

// C = beta D + gamma (K + K^T): tile pairs (i, j) and (j, i), i <= j, one block each pair. D is
// symmetric and read at (i, j) only; C is exactly symmetric. Bound by its bytes (n = 4096: 12 us, 5.6
// TB/s from the caches).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_symmetrise(const T* K, int64_t ldk, int64_t sK,
                                                         const T* D, int64_t ldd, int64_t sD, T* C,
                                                         int64_t ldc, int64_t sC, float beta,
                                                         float gamma) {
  __shared__ float tile[kT][kT + 1];
  // pair index -> (i, j), i <= j: column j holds j + 1 pairs
  const int t = blockIdx.x;
  int j = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while ((j + 1) * (j + 2) / 2 <= t) ++j;
  while (j * (j + 1) / 2 > t) --j;
  const int i = t - j * (j + 1) / 2;
  const int b = blockIdx.y;
  const T* k = K + b * sK;
  T* c = C + b * sC;
  typedef T t4 __attribute__((ext_vector_type(4)));
  const int lx = threadIdx.x % 16 * 4, ly = threadIdx.x / 16;      // 4 columns, 16 rows a pass
  constexpr int Q = kT / 16;
  t4 v[Q], w[Q], d[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int r = ly + 16 * q;
    v[q] = *reinterpret_cast<const t4*>(k + (int64_t)(i * kT + r) * ldk + j * kT + lx);
    w[q] = *reinterpret_cast<const t4*>(k + (int64_t)(j * kT + r) * ldk + i * kT + lx);
    if (D) d[q] = *reinterpret_cast<const t4*>(D + b * sD + (int64_t)(i * kT + r) * ldd + j * kT + lx);
  }
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) tile[ly + 16 * q][lx + e] = (float)w[q][e];
  __syncthreads();
  float o[Q][4];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int r = ly + 16 * q;
    t4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[q][e] = gamma * ((float)v[q][e] + tile[lx + e][r]);
      if (D) o[q][e] += beta * (float)d[q][e];
      x[e] = (T)o[q][e];
    }
    *reinterpret_cast<t4*>(c + (int64_t)(i * kT + r) * ldc + j * kT + lx) = x;
  }
  if (i == j) return;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) tile[ly + 16 * q][lx + e] = o[q][e];
  __syncthreads();
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int r = ly + 16 * q;
    t4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (T)tile[lx + e][r];
    *reinterpret_cast<t4*>(c + (int64_t)(j * kT + r) * ldc + i * kT + lx) = x;
  }
}

// The n x n side of an iteration in one launch, for matrices whose launches count more than their
// arithmetic. C2 = alpha [E; X] [E; X]^T (2 n_p square) holds A = X X^T in its last quarter, K = E X^T
// in its second and K^T in its third. A block makes one 32 x 32 tile of P and of Q,
//   P_ij = a I + b A_ij + c A_i A_j^T,   Q_ij = b S_ij + c (A_i S_j^T + S_i A_j^T),
// from the row blocks A_i, A_j, S_i = K_i + K^T_i, S_j (A and S are symmetric), and writes them as
// the operand of the update: float32
//   [ r P  r Q ; 0  x P ],
// float16, for k_nsb_update,
//   [ r P  r Q ; x P  x dP ; r dP ],   dP = 2^11 (P - its float16 value), all times p.
// In P E + Q X the two terms cancel, which makes P's rounding the largest of an iteration (relative
// error of the gradient at 3 x 1111x333, 1.7e-3 of it the output's own rounding: 2.6e-3 without dP, 2.1e-3
// with it).
// Where X_0 was scaled by a power of two, the first iteration's X is short of the normalised one by
// a factor s in [1, 2): A by s^2 and S by s, and P and Q take s more for the X they multiply.
// The row blocks go through LDS, whole 128-byte lines at a time, and each wave takes a fourth of
// every line (fragments straight from memory touch 32 lines a load: 27 against 16 us on 3 x 512^2).
// Twice the arithmetic of the separate symmetric products, but no intermediate leaves the chip. 14 us
// on 3 x 512^2 (9 on 3 x 333^2, stopping at n), 9 on 256^2 in float32: a launch, and k-tiles of LDS
// fills one after the other.
typedef float floatx16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ void mma32(floatx16& acc, u32x4 a, u32x4 b, _Float16) {
  typedef _Float16 half8 __attribute__((ext_vector_type(8)));
  acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a),
                                               __builtin_bit_cast(half8, b), acc, 0, 0, 0);
}
__device__ __forceinline__ void mma32(floatx16& acc, u32x4 a, u32x4 b, float) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[p]), __uint_as_float(b[p]), acc, 0,
                                               0, 0);
}

struct SquareArgs {
  const void* C2;
  void* PQ;
  int64_t ld, stride;        // of both (elements)
  int n, n_p;
  int tiles;                 // of 32 rows: up to n_p; float16: as far as k_nsb_update reads
  float a, b, c, r, x, p;
  const double* scale;       // k_nsb_scales' (exact), in the first iteration
  double S;
};

template <typename T>
__global__ __launch_bounds__(256) void k_nsb_square(SquareArgs g) {
  constexpr int VEC = 16 / (int)sizeof(T), BK = 8 * VEC, PITCH = 9;      // 16-byte chunks
  typedef T vec __attribute__((ext_vector_type(VEC)));
  __shared__ float part[4][2][16][64];
  __shared__ u32x4 rows[4][32 * PITCH];              // A_i, A_j, S_i, S_j: 128 bytes of 32 rows
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tiles = g.tiles;
  const int i0 = (int)(blockIdx.x / tiles) * 32, j0 = (int)(blockIdx.x % tiles) * 32;
  const T* C2 = static_cast<const T*>(g.C2) + blockIdx.y * g.stride;
  T* PQ = static_cast<T*>(g.PQ) + blockIdx.y * g.stride;
  const int row = lane & 31;
  const T* K = C2 + g.n_p;                         // [E X^T]
  const T* KT = C2 + g.n_p * g.ld;                 // [X E^T]
  const T* A = KT + g.n_p;
  floatx16 pa, qa;
#pragma unroll
  for (int e = 0; e < 16; ++e) pa[e] = qa[e] = 0.f;
  const int lr = threadIdx.x >> 3, lc = threadIdx.x & 7;         // this thread's chunk of a block
  const int64_t oi = (i0 + lr) * g.ld + lc * VEC, oj = (j0 + lr) * g.ld + lc * VEC;
  auto at = [&](const T* base, int64_t o) { return *reinterpret_cast<const vec*>(base + o); };
  vec ai = at(A, oi), aj = at(A, oj), ki = at(K, oi), kj = at(K, oj), ti = at(KT, oi), tj = at(KT, oj);
  // behind n everything is zero: k stops there, and tiles there are written without a product
  const int depth = i0 >= g.n || j0 >= g.n ? 0 : g.n;
  for (int k = 0; k < depth; k += BK) {
    const int o = lr * PITCH + lc;
    rows[0][o] = __builtin_bit_cast(u32x4, ai);
    rows[1][o] = __builtin_bit_cast(u32x4, aj);
    rows[2][o] = __builtin_bit_cast(u32x4, ki + ti);
    rows[3][o] = __builtin_bit_cast(u32x4, kj + tj);
    __syncthreads();
    if (k + BK < depth) {
      const int x = k + BK;
      ai = at(A, oi + x);
      aj = at(A, oj + x);
      ki = at(K, oi + x);
      kj = at(K, oj + x);
      ti = at(KT, oi + x);
      tj = at(KT, oj + x);
    }
    const int f = row * PITCH + 2 * wave + (lane >> 5);
    const u32x4 fai = rows[0][f], faj = rows[1][f], fsi = rows[2][f], fsj = rows[3][f];
    mma32(pa, faj, fai, T{});            // a lane's registers: 4 neighbouring columns of row i
    mma32(qa, fsj, fai, T{});
    mma32(qa, faj, fsi, T{});
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    part[wave][0][e][lane] = pa[e];
    part[wave][1][e][lane] = qa[e];
  }
  __syncthreads();
  // wave w finishes register groups w: columns 8 w + 4 (lane >> 5) .. + 3 of row lane & 31
  typedef T t4 __attribute__((ext_vector_type(4)));
  float b = g.b, c = g.c, s = 1.f;
  if (g.scale) {
    const double* sc = g.scale + 4 * blockIdx.y;
    if (sc[0] > 0.0) s = (float)(sc[1] * g.S / sc[0]);
    b *= s * s;
    c *= s * s * s * s;
  }
  const int i = i0 + row, j = j0 + 8 * wave + 4 * (lane >> 5);
  const t4 av = *reinterpret_cast<const t4*>(A + i * g.ld + j);
  const t4 kv = *reinterpret_cast<const t4*>(K + i * g.ld + j);
  const t4 kt = *reinterpret_cast<const t4*>(KT + i * g.ld + j);
  t4 p1, p2, q, lo, rlo;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int x = 4 * wave + e;
    const float ps = part[0][0][x][lane] + part[1][0][x][lane] + part[2][0][x][lane] + part[3][0][x][lane];
    const float qs = part[0][1][x][lane] + part[1][1][x][lane] + part[2][1][x][lane] + part[3][1][x][lane];
    float p = b * (float)av[e] + c * ps;
    if (i == j + e && i < g.n) p += g.a;
    p *= g.p;
    const float rp = g.r * p, sp = s * g.x * p;
    p1[e] = (T)rp;
    p2[e] = (T)sp;
    rlo[e] = (T)(2048.f * (rp - (float)p1[e]));
    lo[e] = (T)(2048.f * (sp - (float)p2[e]));
    q[e] = (T)(g.r * g.p * (b * (float)(kv[e] + kt[e]) + c * qs));
  }
  T* top = PQ + i * g.ld + j;
  T* low = top + g.n_p * g.ld;
  *reinterpret_cast<t4*>(top) = p1;
  *reinterpret_cast<t4*>(top + g.n_p) = q;
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<t4*>(low) = p2;
    *reinterpret_cast<t4*>(low + g.n_p) = lo;
    *reinterpret_cast<t4*>(low + g.n_p * g.ld) = rlo;
  } else {
    *reinterpret_cast<t4*>(low) = t4{};
    *reinterpret_cast<t4*>(low + g.n_p) = p2;
  }
}

// C2's blocks A, K and K^T for short reductions, float16: 64 x 64 tiles of E X^T and of half of X X^T,
// each stored in both places; as far as k_nsb_square reads (n to the next 128; zeros behind n). Eight
// waves in two groups of four, 32 x 32 a wave, the groups taking k-tiles of 64 in turn: half as many
// steps one after the other, which are what bounds it; their sums are added through LDS. Each group
// has a ring of four LDS stages that DMA fills. 9 us on 3 x 1111x333, 18 on the general product and its
// tail (the whole call, T = 5, without dX: 201 / 246; 2 x 257x300 142 / 170, 512x8192 398 / 394, 8 x 512x512 410 / 386).
struct GramArgs {
  const _Float16* V;         // [E; X]
  int64_t ldv, sV;
  _Float16* C2;
  int64_t ld, stride;
  int n, n_p, row_tiles;     // row_tiles: of 64, up to n rounded up to 128
  int64_t m;
  float alpha;
};

__global__ __launch_bounds__(512) void k_nsb_gram(GramArgs g) {
  constexpr int NS = 4, TILE = 64 * kChunks, STAGE = 2 * TILE, GROUP = NS * STAGE, TP = 72;
  __shared__ u32x4 lds[2 * GROUP];                   // 128 KB
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave8 = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = wave8 >> 2, wave = wave8 & 3, wm = wave >> 1, wn = wave & 1;
  const int rt = g.row_tiles, unit = (int)blockIdx.x;
  const bool cross = unit < rt * rt;
  int ti, tj;
  if (cross) {
    ti = unit / rt;
    tj = unit % rt;
  } else {                                           // row by row of the upper half
    int left = unit - rt * rt;
    ti = 0;
    while (left >= rt - ti) left -= rt - ti++;
    tj = ti + left;
  }
  const int i0 = (cross ? 0 : g.n_p) + ti * 64, j0 = g.n_p + tj * 64;      // rows of V
  const int KL = ti * 64 >= g.n || tj * 64 >= g.n ? 0 : ((int)g.m + 63) / 64;
  const int ldv = (int)g.ldv;
  const int64_t b = blockIdx.y;

  floatx16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  if (KL > 0) {
    const __amdgpu_buffer_rsrc_t rV = make_rsrc(g.V + b * g.sV, (int64_t)2 * g.n_p * g.ldv * 2);
    const __amdgpu_buffer_rsrc_t none = make_rsrc(g.V, 0);     // reads zeros from nowhere
    u32x4* ring = lds + group * GROUP;
    int off[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (wave * 2 + i) * 8 + (lane >> 3);
      off[i] = (row * ldv + 8 * ((lane & 7) ^ ((row ^ ((row >> 3) & 3)) & 7))) * 2;
    }
    auto issue = [&](int step, int st) {
      const int kt = 2 * step + group;
      const bool real = kt < KL;
      const __amdgpu_buffer_rsrc_t r = real ? rV : none;
      const int oa = real ? (i0 * ldv + kt * 64) * 2 : 0, ob = real ? (j0 * ldv + kt * 64) * 2 : 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        dma16(r, &ring[st * STAGE + (wave * 2 + i) * 64], off[i], oa);
        dma16(r, &ring[st * STAGE + TILE + (wave * 2 + i) * 64], off[i], ob);
      }
    };
    const int steps = (KL + 1) / 2;
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) issue(s, s);
    int st = 0, fill = NS - 1;
    for (int step = 0; step < steps; ++step) {
      // as in k_nsb_update: this step's k-tiles have landed, the stage before is free
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0070 | (NS - 2) * 4);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      issue(step + NS - 1, fill);
      const u32x4* A = ring + st * STAGE;
      const u32x4* B = A + TILE;
      u32x4 a[4], v[4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int ch = 2 * ks + (lane >> 5);
        a[ks] = A[swz(wm * 32 + (lane & 31), ch)];
        v[ks] = B[swz(wn * 32 + (lane & 31), ch)];
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) mma32(acc, v[ks], a[ks], _Float16{});
      st = st + 1 == NS ? 0 : st + 1;
      fill = fill + 1 == NS ? 0 : fill + 1;
    }
    block_sync();                 // no DMA is in flight
    float(*sums)[16][64] = reinterpret_cast<float(*)[16][64]>(lds);
    if (group == 1) {
#pragma unroll
      for (int e = 0; e < 16; ++e) sums[wave][e][lane] = acc[e];
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] = (acc[e] + sums[wave][e][lane]) * g.alpha;
    }
    __syncthreads();
  }
  // a lane's registers: 4 neighbouring columns of one row, in 4 groups; transposed through LDS
  typedef _Float16 half4 __attribute__((ext_vector_type(4)));
  _Float16* C2 = g.C2 + b * g.stride;
  _Float16* T = reinterpret_cast<_Float16*>(lds);
  if (group == 0) {
    const int r = wm * 32 + (lane & 31), c = wn * 32 + 4 * (lane >> 5);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      half4 h;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = (_Float16)acc[4 * q + e];
        T[(c + 8 * q + e) * TP + r] = h[e];
      }
      *reinterpret_cast<half4*>(C2 + (i0 + r) * g.ld + j0 + c + 8 * q) = h;
    }
  }
  __syncthreads();
  if (!cross && ti == tj) return;
  const int row = tid >> 3, ch = tid & 7;
  *reinterpret_cast<u32x4*>(C2 + (j0 + row) * g.ld + i0 + 8 * ch) =
      *reinterpret_cast<const u32x4*>(T + row * TP + 8 * ch);
}

// The update of that form, float16:
//   E' = r P E + r Q X,   X' = P X,   P, and X within its own update, as two float16 numbers (dX = 2^11 (X
// less its float16 value), a third block of V; none in the first iteration): X's rounding, carried
// from one iteration to the next, is what low-rank matrices amplify (2 x 284x1083, rank 64 plus noise:
// 2.8e-3 with one, 1.8e-3 with two, 1.7e-3 of it the output's own).
// Tiles of BT x BT (128: eight waves of 32 x 64; 64, where there are few tiles: four of 32 x 32),
// k-tiles of 64 in a ring of four LDS stages that DMA fills, one barrier each; operands as in
// grouped.hip's ring kernel (V is read along the output, through the transposing LDS load). The
// small parts come first and are scaled down before the rest is added. Tiles of the padding are
// zeros, without a product, and the k-tiles stop at n. TRANS (the last iteration of tall matrices): E'
// alone, transposed. 19 us on 3 x 1111x333 (18 dependent k-tiles of about 0.7 us; the padded
// product on the general GEMM, one part of P, 14 us and 7 for joining its parts).
struct UpdateArgs {
  const _Float16* PQ;        // of k_nsb_square, 3 n_p rows
  int64_t ld, stride;
  const _Float16* V;         // [E; X; dX]
  int64_t ldv, sV;
  _Float16* out;             // [E'; X'; dX'], or E'^T
  int64_t ldo, sO;
  int n, n_p;
  int64_t m;
  int row_tiles, col_tiles, columns;   // row tiles of E' and X'; columns of tiles of all matrices
  int first;                 // no dX
  float inv;                 // 1 / p
};

template <int BT, bool TRANS>
__global__ __launch_bounds__(4 * BT) void k_nsb_update(UpdateArgs g) {
  constexpr int NS = 4, STAGE = 2 * BT * kChunks, KROW = 2 * BT, FN = BT / 64, KCH = BT / 8;
  __shared__ u32x4 lds[NS * STAGE];                  // 128 or 64 KB
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  // Blocks go round the 8 XCDs one by one: all row tiles of a column of tiles on one of them, which
  // then reads that part of V alone.
  const int row_tiles = g.n_p / BT, all = g.row_tiles, place = (int)blockIdx.x >> 3;
  const int column = ((int)blockIdx.x & 7) + 8 * (place / all), down = place % all;
  if (column >= g.columns) return;
  const bool x_rows = down >= row_tiles;
  const int i0 = (down - (x_rows ? row_tiles : 0)) * BT, j0 = column % g.col_tiles * BT;
  const int64_t b = column / g.col_tiles;
  const int per = (g.n + 63) / 64;                   // k-tiles of a product of depth n
  const int KL = i0 >= g.n || j0 >= g.m ? 0 : x_rows && g.first ? 2 * per : 3 * per;
  const int small = x_rows && !g.first ? 2 * per : per;        // k-tiles of the small parts
  const int ld = (int)g.ld, ldv = (int)g.ldv;

  floatx16 acc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[j][e] = 0.f;
  if (KL > 0) {
    const __amdgpu_buffer_rsrc_t rA =
        make_rsrc(g.PQ + b * g.stride, (int64_t)3 * g.n_p * g.ld * 2);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.V + b * g.sV, (int64_t)3 * g.n_p * g.ldv * 2);
    const __amdgpu_buffer_rsrc_t none = make_rsrc(g.PQ, 0);    // reads zeros from nowhere
    int offA[2], offB[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (wave * 2 + i) * 8 + (lane >> 3);
      offA[i] = (row * ld + 8 * ((lane & 7) ^ ((row ^ ((row >> 3) & 3)) & 7))) * 2;
      const int kr = (wave * 2 + i) * (64 / KCH) + lane / KCH;
      const int x = BT == 128 ? 4 * (kr & 3) : 4 * ((kr >> 1) & 1);
      offB[i] = (kr * ldv + 8 * ((lane % KCH) ^ x)) * 2;
    }
    auto issue = [&](int kt, int st) {
      const bool real = kt < KL;
      const __amdgpu_buffer_rsrc_t a = real ? rA : none, v = real ? rB : none;
      // E': r dP E, r P E, r Q X; X': dP X, P dX (not in the first iteration), P X
      const int seg = kt >= 2 * per ? 2 : kt >= per ? 1 : 0;
      const int k = (kt - seg * per) * 64;
      const int ar = x_rows ? g.n_p : seg == 0 ? 2 * g.n_p : 0;
      const int ac = x_rows ? (seg == 0 ? g.n_p : 0) : seg == 2 ? g.n_p : 0;
      const int vr = x_rows ? (seg == 1 && !g.first ? 2 * g.n_p : g.n_p) : seg == 2 ? g.n_p : 0;
      const int oa = real ? ((ar + i0) * ld + ac + k) * 2 : 0;
      const int ov = real ? ((vr + k) * ldv + j0) * 2 : 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        dma16(v, &lds[st * STAGE + BT * kChunks + (wave * 2 + i) * 64], offB[i], ov);
        dma16(a, &lds[st * STAGE + (wave * 2 + i) * 64], offA[i], oa);
      }
    };
    const int G = lane >> 4, kb = 8 * (G >> 1) + ((lane & 15) >> 2);
    const int x = BT == 128 ? 4 * (kb & 3) : 4 * ((kb >> 1) & 1);
    uint32_t b_addr[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int col = wn * (BT / 2) + 32 * j + 16 * (G & 1) + 4 * (lane & 3);
      b_addr[j] = lds_address(lds) + BT * 128 + kb * KROW + ((col >> 3) ^ x) * 16 +
                  (col & 7) * 2;
    }
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) issue(s, s);
    int st = 0, fill = NS - 1;
    for (int kt = 0; kt < KL; ++kt) {
      // k-tile kt has landed (two newer ones, eight DMAs, may be on their way), for every wave
      // behind the barrier, where the stage of k-tile kt - 1 is free too
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x0070 | (NS - 2) * 4);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      issue(kt + NS - 1, fill);
      const u32x4* A = lds + st * STAGE;
      u32x4 a[4], v[4][FN];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) a[ks] = A[swz(wm * 32 + (lane & 31), 2 * ks + (lane >> 5))];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        // waited for in the same block (the compiler would wait for every outstanding DMA)
        u32x2 t[8];
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8\n\t"
            "ds_read_b64_tr_b16 %1, %8 offset:%c9\n\t"
            "ds_read_b64_tr_b16 %2, %8 offset:%c10\n\t"
            "ds_read_b64_tr_b16 %3, %8 offset:%c11\n\t"
            "ds_read_b64_tr_b16 %4, %8 offset:%c12\n\t"
            "ds_read_b64_tr_b16 %5, %8 offset:%c13\n\t"
            "ds_read_b64_tr_b16 %6, %8 offset:%c14\n\t"
            "ds_read_b64_tr_b16 %7, %8 offset:%c15\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3]), "=&v"(t[4]), "=&v"(t[5]),
              "=&v"(t[6]), "=&v"(t[7])
            : "v"(b_addr[j] + (uint32_t)(st * STAGE * 16)), "i"(4 * KROW), "i"(16 * KROW),
              "i"(20 * KROW), "i"(32 * KROW), "i"(36 * KROW), "i"(48 * KROW), "i"(52 * KROW));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          v[ks][j] = u32x4{t[2 * ks].x, t[2 * ks].y, t[2 * ks + 1].x, t[2 * ks + 1].y};
      }
      if (kt == small) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[j][e] *= 0x1p-11f;
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if constexpr (TRANS) mma32(acc[j], a[ks], v[ks][j], _Float16{});
          else mma32(acc[j], v[ks][j], a[ks], _Float16{});
        }
      st = st + 1 == NS ? 0 : st + 1;
      fill = fill + 1 == NS ? 0 : fill + 1;
    }
    block_sync();                 // no DMA is in flight when the block ends
  }
  // a lane's registers: 4 neighbouring columns of one row (TRANS: rows of one column) in 4 groups
  typedef _Float16 half4 __attribute__((ext_vector_type(4)));
  const int one = lane & 31, four = 4 * (lane >> 5);
  _Float16* out = g.out + b * g.sO;
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int r = i0 + wm * 32, c = j0 + wn * (BT / 2) + 32 * j;
    _Float16* o = out + (TRANS ? (c + one) * g.ldo + r + four
                               : ((x_rows ? g.n_p : 0) + r + one) * g.ldo + c + four);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      half4 h, d;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = acc[j][4 * q + e] * g.inv;
        h[e] = (_Float16)v;
        d[e] = (_Float16)(2048.f * (v - (float)h[e]));
      }
      *reinterpret_cast<half4*>(o + 8 * q) = h;
      if (x_rows) *reinterpret_cast<half4*>(o + g.n_p * g.ldo + 8 * q) = d;
    }
  }
}

// ---- short sides up to 64 -------------------------------------------------------------------
//
// The n x n side of such a matrix fits one block, so an iteration is one launch: every block of a
// matrix adds the partial Gram matrices A and K that all its blocks left, forms P and Q from them
// by itself, updates its own columns of E and X (64 at a time, in place) and leaves the next
// partial sums from the new values while it has them. float32 throughout; matrices padded to 64
// rows, not 256. Bound by the latency of its few dependent products; with T = 5, against the form of
// three launches: 64x256 104 / 194 us, 24 x 64x1024 234 / 1255, 24 x 64x12288 971 / 7481. The four
// waves own the quadrants of every 64 x 64 product.
constexpr int kN = 64, kNP = kN + 1;          // LDS row pitch: 32 rows of one column on 32 banks

// acc (quadrant qi, qj) += sum over k < 64 of L[i ls + k lk] R[j rs + k rk]
__device__ __forceinline__ void quad64(floatx16& acc, const float* L, int ls, int lk, const float* R,
                                       int rs, int rk, int qi, int qj) {
  const int lane = threadIdx.x & 63, k1 = lane >> 5;
  const float* l = L + (32 * qi + (lane & 31)) * ls + k1 * lk;
  const float* r = R + (32 * qj + (lane & 31)) * rs + k1 * rk;
#pragma unroll 8
  for (int k = 0; k < kN; k += 2)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(l[k * lk], r[k * rk], acc, 0, 0, 0);
}
// element e of a lane: row, column within the 64 x 64 result
__device__ __forceinline__ int quad_row(int e, int qi) {
  return 32 * qi + 8 * (e / 4) + 4 * ((threadIdx.x & 63) >> 5) + e % 4;
}
__device__ __forceinline__ int quad_col(int qj) { return 32 * qj + (threadIdx.x & 31); }
__device__ __forceinline__ floatx16 zero16() {
  floatx16 z;
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] = 0.f;
  return z;
}

struct SmallArgs {
  float* V;                // [E; X] per matrix: 128 rows, pitch ld
  float* part[2];          // [matrix][block][A, K][64 x 64], read and written in turn
  float* Et;               // last step of a tall matrix: E^T, m x 64
  int64_t ld, v_stride, et_stride;
  int n, cols_per, blocks;   // columns and blocks per matrix
  int64_t m;
};

__device__ __forceinline__ float* part_of(const SmallArgs& g, int parity, int b, int blk) {
  return g.part[parity] + ((int64_t)b * g.blocks + blk) * (2 * kN * kN);
}

__device__ __forceinline__ void leave_parts(const SmallArgs& g, int parity, const floatx16& aa,
                                            const floatx16& kk, int qi, int qj) {
  float* out = part_of(g, parity, blockIdx.y, blockIdx.x);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int o = quad_row(e, qi) * kN + quad_col(qj);
    out[o] = aa[e];
    out[kN * kN + o] = kk[e];
  }
}

// E_0, X_0 from dO and X (rows x cols as stored; tall: the transposed tile), and their partial sums.
template <typename TX>
__global__ __launch_bounds__(256) void k_nsb_small_load(const TX* X, const TX* G, bool tall,
                                                        const double* scale, SmallArgs g) {
  __shared__ float tile[2][kN * kNP];
  const int b = blockIdx.y, wave = threadIdx.x >> 6, qi = wave >> 1, qj = wave & 1;
  const int64_t c_begin = (int64_t)blockIdx.x * g.cols_per;
  const int64_t c_end = c_begin + g.cols_per < g.ld ? c_begin + g.cols_per : g.ld;
  floatx16 aa = zero16(), kk = zero16();
  for (int64_t c0 = c_begin; c0 < c_end; c0 += kN) {
    for (int which = 0; which < 2; ++which) {
      const TX* src = (which ? X : G) + (int64_t)b * g.n * g.m;
      const double sc = scale[4 * b + (which ? 0 : 2)];
      for (int q = threadIdx.x; q < kN * kN; q += 256) {
        // lanes run along the stored rows
        const int i = tall ? q % kN : q / kN, c = tall ? q / kN : q % kN;
        float v = 0.f;
        if (i < g.n && c0 + c < g.m) {
          const int64_t o = tall ? (c0 + c) * g.n + i : i * g.m + c0 + c;
          v = (float)((double)widen(src[o]) * sc);
        }
        tile[which][i * kNP + c] = v;
      }
    }
    __syncthreads();
    float* V = g.V + b * g.v_stride + c0;
    for (int q = threadIdx.x; q < 2 * kN * kN; q += 256) {
      const int r = q / kN, c = q % kN;
      V[r * g.ld + c] = tile[r / kN][(r % kN) * kNP + c];
    }
    quad64(aa, tile[1], kNP, 1, tile[1], kNP, 1, qi, qj);
    quad64(kk, tile[0], kNP, 1, tile[1], kNP, 1, qi, qj);
    __syncthreads();
  }
  leave_parts(g, 0, aa, kk, qi, qj);
}

// xr: the new X's scale over the old one's, a power of two
__global__ __launch_bounds__(256) void k_nsb_small_step(SmallArgs g, float a, float bb, float c,
                                                        float xr, int parity, bool last) {
  __shared__ float P[kN * kNP], Q[kN * kNP], E[kN * kNP], X[kN * kNP];
  const int b = blockIdx.y, tid = threadIdx.x, wave = tid >> 6, qi = wave >> 1, qj = wave & 1;
  {
    // A and K: the blocks' partial sums, in block order
    float4 s[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] = float4{0.f, 0.f, 0.f, 0.f};
    const float4* src = reinterpret_cast<const float4*>(part_of(g, parity, b, 0)) + tid;
#pragma unroll 2
    for (int blk = 0; blk < g.blocks; ++blk, src += 2 * kN * kN / 4) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 v = src[256 * q];
        s[q].x += v.x;
        s[q].y += v.y;
        s[q].z += v.z;
        s[q].w += v.w;
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int o = (tid + 256 * (q & 3)) * 4;
      float* dst = (q < 4 ? P : Q) + (o / kN) * kNP + o % kN;
      dst[0] = s[q].x;
      dst[1] = s[q].y;
      dst[2] = s[q].z;
      dst[3] = s[q].w;
    }
  }
  __syncthreads();
  // S = K + K^T, in Q
  float sv[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = quad_row(e, qi), j = quad_col(qj);
    sv[e] = Q[i * kNP + j] + Q[j * kNP + i];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 16; ++e) Q[quad_row(e, qi) * kNP + quad_col(qj)] = sv[e];
  __syncthreads();
  floatx16 a2 = zero16(), as = zero16();
  quad64(a2, P, kNP, 1, P, kNP, 1, qi, qj);
  quad64(as, P, kNP, 1, Q, kNP, 1, qi, qj);
#pragma unroll
  for (int e = 0; e < 16; ++e) E[quad_row(e, qi) * kNP + quad_col(qj)] = as[e];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int i = quad_row(e, qi), j = quad_col(qj);
    a2[e] = c * a2[e] + bb * P[i * kNP + j] + (i == j && i < g.n ? a : 0.f);
    as[e] = bb * sv[e] + c * (as[e] + E[j * kNP + i]);
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int o = quad_row(e, qi) * kNP + quad_col(qj);
    P[o] = a2[e];
    Q[o] = as[e];
  }
  floatx16 aa = zero16(), kk = zero16();
  const int64_t c_begin = (int64_t)blockIdx.x * g.cols_per;
  const int64_t c_end = c_begin + g.cols_per < g.ld ? c_begin + g.cols_per : g.ld;
  for (int64_t c0 = c_begin; c0 < c_end; c0 += kN) {
    float* V = g.V + b * g.v_stride + c0;
    for (int q = tid; q < 2 * kN * kN / 4; q += 256) {
      const int r = q / (kN / 4), x = q % (kN / 4) * 4;
      const float4 v = *reinterpret_cast<const float4*>(V + r * g.ld + x);
      float* dst = (r < kN ? E : X) + (r % kN) * kNP + x;
      dst[0] = v.x;
      dst[1] = v.y;
      dst[2] = v.z;
      dst[3] = v.w;
    }
    __syncthreads();
    floatx16 en = zero16(), xn = zero16();
    quad64(en, P, kNP, 1, E, 1, kNP, qi, qj);
    quad64(en, Q, kNP, 1, X, 1, kNP, qi, qj);
    if (!last) quad64(xn, P, kNP, 1, X, 1, kNP, qi, qj);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int i = quad_row(e, qi), j = quad_col(qj);
      xn[e] *= xr;
      E[i * kNP + j] = en[e];
      X[i * kNP + j] = xn[e];
      if (!last || !g.Et) V[i * g.ld + j] = en[e];
      if (!last) V[(kN + i) * g.ld + j] = xn[e];
    }
    __syncthreads();
    if (!last) {
      quad64(aa, X, kNP, 1, X, kNP, 1, qi, qj);
      quad64(kk, E, kNP, 1, X, kNP, 1, qi, qj);
    } else if (g.Et) {
      float* Et = g.Et + b * g.et_stride + c0 * kN;
      for (int q = tid; q < kN * kN; q += 256) {
        const int col = q / kN, i = q % kN;
        if (c0 + col < g.m) Et[q] = E[i * kNP + col];
      }
    }
    __syncthreads();
  }
  if (!last) leave_parts(g, parity ^ 1, aa, kk, qi, qj);
}

// Partial sums of <X, E> (E in the stored layout, padded rows), float64: block x of nblk takes
// rows x, x + nblk, ... Bound by its bytes (8 x 1024x8192: 51 us, 5.3 TB/s).
template <typename TX, typename TE>
__global__ __launch_bounds__(kThreads) void k_nsb_dot(const TX* X, const TE* E, int64_t rows,
                                                      int64_t cols, int64_t ld, int64_t sE,
                                                      double* part) {
  __shared__ double red[kThreads];
  const int b = blockIdx.y;
  double s = 0.0;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const TX* x = X + ((int64_t)b * rows + r) * cols;
    const TE* e = E + b * sE + r * ld;
    if (cols % 8 == 0) {
      for (int64_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
        float xv[8], ev[8];
        load8(x + c, xv);
        load8(e + c, ev);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (double)xv[i] * (double)ev[i];
      }
    } else {
      for (int64_t c = threadIdx.x; c < cols; c += kThreads)
        s += (double)widen(x[c]) * (double)(float)e[c];
    }
  }
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) part[(int64_t)b * gridDim.x + blockIdx.x] = red[0];
}

// dX = (E - X_0 <X_0, E>) / ||X|| with E = E_T ||dO|| / eT: float64 arithmetic (norms of any
// float32 range, one rounding at the end; the pass is bound by its bytes: 8 x 1024x8192 66 us, 6.1
// TB/s).
template <typename TX, typename TE>
__global__ __launch_bounds__(kThreads) void k_nsb_project(const TX* X, const TE* E, int64_t rows,
                                                          int64_t cols, int64_t ld, int64_t sE,
                                                          const double* part, int nblk,
                                                          const double* scale, double inv_eT,
                                                          TX* out) {
  __shared__ double red[kThreads];
  const int b = blockIdx.y;
  double s = 0.0;
  for (int i = threadIdx.x; i < nblk; i += kThreads) s += part[(int64_t)b * nblk + i];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  const double ix = scale[4 * b + 1], fe = scale[4 * b + 3] * inv_eT * ix;
  const double cx = -red[0] * ix * ix * fe;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const TX* x = X + ((int64_t)b * rows + r) * cols;
    const TE* e = E + b * sE + r * ld;
    TX* o = out + ((int64_t)b * rows + r) * cols;
    if (cols % 8 == 0) {
      for (int64_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
        float xv[8], ev[8];
        load8(x + c, xv);
        load8(e + c, ev);
        TX ov[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) narrow((double)ev[i] * fe + (double)xv[i] * cx, &ov[i]);
        store8(o + c, ov);
      }
    } else {
      for (int64_t c = threadIdx.x; c < cols; c += kThreads)
        narrow((double)(float)e[c] * fe + (double)widen(x[c]) * cx, &o[c]);
    }
  }
}

hipError_t last() { return hipGetLastError(); }

}  // namespace

hipError_t nsb_scales(const double* px, const double* pg, int nblk, int count, double S, double e0,
                      bool exact, double* scale, hipStream_t s) {
  hipLaunchKernelGGL(k_nsb_scales, dim3(count), dim3(kThreads), 0, s, px, pg, nblk, S, e0, exact,
                     scale);
  return last();
}

hipError_t nsb_load(const void* X, const void* G, Store st, int count, int64_t rows, int64_t cols,
                    const double* scale, Elem e, int64_t rows_p, int64_t cols_p,
                    const NsbDst& straight, const NsbDst& transposed, hipStream_t s) {
  const dim3 grid((unsigned)(cols_p / kT), (unsigned)(rows_p / kT), 2 * count);
  const LoadDst a{straight.p, straight.ld, straight.stride, straight.offset};
  const LoadDst t{transposed.p, transposed.ld, transposed.stride, transposed.offset};
  const int64_t n = rows * cols;
  // a transposed layout goes through LDS tiles; the straight one alone is a row pass (134 M elements
  // of 4096 x 16384: 284 against 81 us)
  const dim3 flat((unsigned)((cols_p / 8 + 4 * kThreads - 1) / (4 * kThreads)), (unsigned)rows_p,
                  2 * count);
#define MNS_NSB_LOAD(TX, TO)                                                                \
  do {                                                                                      \
    if (t.p)                                                                                \
      hipLaunchKernelGGL((k_nsb_load<TX, TO>), grid, dim3(kThreads), 0, s,                  \
                         static_cast<const TX*>(X), static_cast<const TX*>(G), rows, cols,  \
                         n, scale, a, t);                                                   \
    else                                                                                    \
      hipLaunchKernelGGL((k_nsb_load_rows<TX, TO>), flat, dim3(kThreads), 0, s,             \
                         static_cast<const TX*>(X), static_cast<const TX*>(G), rows, cols,  \
                         cols_p, n, scale, a);                                              \
  } while (0)
  if (st == Store::F32) MNS_NSB_LOAD(float, float);
  else if (e == Elem::F32) MNS_NSB_LOAD(uint16_t, float);
  else MNS_NSB_LOAD(uint16_t, _Float16);
#undef MNS_NSB_LOAD
  return last();
}

hipError_t symmetrise(const void* K, int64_t ldk, int64_t sK, const void* D, int64_t ldd,
                      int64_t sD, void* C, int64_t ldc, int64_t sC, Elem e, int count, int64_t n_p,
                      float beta, float gamma, hipStream_t s) {
  const int t = (int)(n_p / kT);
  const dim3 grid(t * (t + 1) / 2, count);
  if (e == Elem::F16)
    hipLaunchKernelGGL(k_symmetrise<_Float16>, grid, dim3(kThreads), 0, s,
                       static_cast<const _Float16*>(K), ldk, sK, static_cast<const _Float16*>(D),
                       ldd, sD, static_cast<_Float16*>(C), ldc, sC, beta, gamma);
  else
    hipLaunchKernelGGL(k_symmetrise<float>, grid, dim3(kThreads), 0, s,
                       static_cast<const float*>(K), ldk, sK, static_cast<const float*>(D), ldd,
                       sD, static_cast<float*>(C), ldc, sC, beta, gamma);
  return last();
}

hipError_t nsb_square(const void* C2, void* PQ, int64_t ld, int64_t stride, Elem e, int count, int n,
                      int n_p, float a, float b, float c, float r, float x, float p,
                      const double* scale, double S, hipStream_t s) {
  const int tiles = (e == Elem::F16 ? (n + 127) / 128 * 128 : n_p) / 32;
  const SquareArgs g{C2, PQ, ld, stride, n, n_p, tiles, a, b, c, r, x, p, scale, S};
  const dim3 grid(tiles * tiles, count);
  if (e == Elem::F16) hipLaunchKernelGGL(k_nsb_square<_Float16>, grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL(k_nsb_square<float>, grid, dim3(256), 0, s, g);
  return last();
}

hipError_t nsb_gram(const void* V, int64_t ldv, int64_t sV, void* C2, int64_t ld, int64_t stride,
                    int count, int n, int n_p, int64_t m, float alpha, hipStream_t s) {
  const int rt = (n + 127) / 128 * 2;
  const GramArgs g{static_cast<const _Float16*>(V), ldv, sV, static_cast<_Float16*>(C2), ld, stride, n,
                   n_p, rt, m, alpha};
  hipLaunchKernelGGL(k_nsb_gram, dim3(rt * rt + rt * (rt + 1) / 2, count), dim3(512), 0, s, g);
  return last();
}

hipError_t nsb_update(const void* PQ, int64_t ld, int64_t stride, const void* V, int64_t ldv,
                      int64_t sV, void* out, int64_t ldo, int64_t sO, int count, int n, int n_p,
                      int64_t m, int64_t m_p, float inv, bool first, bool only_e, bool trans,
                      hipStream_t s) {
  // 64 x 64 where the products fill at most 100 tiles of 128 x 128 (the whole call, T = 5, before dX and
  // k_nsb_gram, us, 64 / 128:
  // 512x512 173 / 208, three of them 234 / 246, 333x1111 184 / 199; two of those, 108 tiles, 244 / 238,
  // 2 x 512x2048 315 / 283)
  const int64_t live = (int64_t)((n + 127) / 128) * ((m + 127) / 128) * 2 * count;
  const int bt = live <= 100 ? 64 : 128;
  const int rt = n_p / bt * (only_e ? 1 : 2), ct = (int)(m_p / bt);
  const UpdateArgs g{static_cast<const _Float16*>(PQ), ld, stride, static_cast<const _Float16*>(V),
                     ldv, sV, static_cast<_Float16*>(out), ldo, sO, n, n_p, m, rt, ct, ct * count,
                     first, inv};
  const dim3 grid((unsigned)((ct * count + 7) / 8 * 8 * rt)), block(4 * bt);
  if (bt == 64) {
    if (trans) hipLaunchKernelGGL((k_nsb_update<64, true>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((k_nsb_update<64, false>), grid, block, 0, s, g);
  } else {
    if (trans) hipLaunchKernelGGL((k_nsb_update<128, true>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((k_nsb_update<128, false>), grid, block, 0, s, g);
  }
  return last();
}

static SmallArgs small_args(const NsbSmall& d) {
  SmallArgs g;
  g.V = d.V;
  g.part[0] = d.part[0];
  g.part[1] = d.part[1];
  g.Et = d.tall ? d.Et : nullptr;
  g.ld = d.ld;
  g.v_stride = 2 * kN * d.ld;
  g.et_stride = d.m * kN;
  g.n = (int)d.n;
  g.cols_per = d.cols_per;
  g.blocks = d.blocks;
  g.m = d.m;
  return g;
}

hipError_t nsb_small_load(const NsbSmall& d, const void* X, const void* G, Store st,
                          const double* scale, hipStream_t s) {
  const dim3 grid(d.blocks, d.count);
  if (st == Store::F32)
    hipLaunchKernelGGL(k_nsb_small_load<float>, grid, dim3(256), 0, s, static_cast<const float*>(X),
                       static_cast<const float*>(G), d.tall, scale, small_args(d));
  else
    hipLaunchKernelGGL(k_nsb_small_load<uint16_t>, grid, dim3(256), 0, s,
                       static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(G), d.tall,
                       scale, small_args(d));
  return last();
}

hipError_t nsb_small_step(const NsbSmall& d, int t, bool last_step, float a, float b, float c,
                          float x, hipStream_t s) {
  hipLaunchKernelGGL(k_nsb_small_step, dim3(d.blocks, d.count), dim3(256), 0, s, small_args(d), a, b,
                     c, x, t & 1, last_step);
  return last();
}

int nsb_dot_blocks(int64_t rows) { return (int)(rows < 512 ? rows : 512); }

hipError_t nsb_finish(const void* X, Store st, const void* E, Elem e, int count, int64_t rows,
                      int64_t cols, int64_t ld, int64_t sE, double* part, const double* scale,
                      double inv_eT, void* out, hipStream_t s) {
  const int nblk = nsb_dot_blocks(rows);
  const dim3 dot(nblk, count), proj((unsigned)(rows < 2048 ? rows : 2048), count);
#define MNS_NSB_FINISH(TX, TE)                                                                  \
  do {                                                                                          \
    hipLaunchKernelGGL((k_nsb_dot<TX, TE>), dot, dim3(kThreads), 0, s, static_cast<const TX*>(X), \
                       static_cast<const TE*>(E), rows, cols, ld, sE, part);                    \
    const hipError_t err = last();                                                              \
    if (err != hipSuccess) return err;                                                          \
    hipLaunchKernelGGL((k_nsb_project<TX, TE>), proj, dim3(kThreads), 0, s,                     \
                       static_cast<const TX*>(X), static_cast<const TE*>(E), rows, cols, ld, sE, \
                       part, nblk, scale, inv_eT, static_cast<TX*>(out));                       \
  } while (0)
  if (st == Store::F32) MNS_NSB_FINISH(float, float);
  else if (e == Elem::F32) MNS_NSB_FINISH(uint16_t, float);
  else MNS_NSB_FINISH(uint16_t, _Float16);
#undef MNS_NSB_FINISH
  return last();
}

}  // namespace mns
