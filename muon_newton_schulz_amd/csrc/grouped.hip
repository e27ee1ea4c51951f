// Products grouped by expert: rows of one token matrix, sorted by expert, against that expert's
// own weight matrix, with group sizes that only the device knows.
//
//   forward          Y_e  = X_e W_e^T        (k_grouped<..., NT>)
//   input gradient   dX_e = dY_e W_e         (k_grouped<..., NN>)
//   weight gradient  G_e  = beta C_e + dY_e^T X_e, reduced over the expert's rows (TN)
//
// Expert e owns rows [offsets[e], offsets[e + 1]) of the token matrices. The offsets are read by
// the kernels only: no host copy, no synchronisation, so the calls can be captured. Every offset
// is clamped to [0, total_rows] and an end before its begin is an empty group, so wrong offsets
// give wrong results but never an access outside the buffers.
#include "mns_internal.h"

#include <type_traits>

namespace mns {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

enum Form { NT = 0, NN = 1, TN = 2 };

struct GroupedArgs {
  const void* A; const void* B; const void* D; void* C;
  int64_t lda, ldb, ldc;        // row pitches, elements (ldc: of C and D)
  int64_t sB, sC;               // per-expert strides of W (NT, NN) and of C, D (TN)
  const int64_t* offsets;
  int64_t total_rows;
  int groups;
  int N, K;                     // NT, NN: output columns and reduction; TN: output rows, columns
  int tiles_n;
  int fill_rest;                // NT, NN: rows of no expert are written as zeros
  float beta;                   // TN
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// Rows [lo, hi) of expert e.
__device__ __forceinline__ void expert_rows(const GroupedArgs& p, int e, int64_t& lo, int64_t& hi) {
  lo = clamp64(p.offsets[e], 0, p.total_rows);
  hi = clamp64(p.offsets[e + 1], lo, p.total_rows);
}

// Row tile `mt` of the list that walks the experts in order, each cut into tiles of BM rows (with
// fill_rest, the rows before the first expert and behind the last one come first and last, as
// expert -1): its expert, first row and the end of the expert's rows. False past the last tile.
// One wave reads 64 experts' bounds at a time and adds their tile counts by a shuffle scan, so
// every wave finds its tile by itself, without a launch or a barrier.
__device__ __forceinline__ bool find_row_tile(const GroupedArgs& p, int BM, int64_t mt, int& expert,
                                              int64_t& row0, int64_t& row_end) {
  const int lane = threadIdx.x & 63;
  const int front = p.fill_rest ? 1 : 0;
  const int count = p.groups + 2 * front;
  int64_t before = 0;
  for (int g0 = 0; g0 < count; g0 += 64) {
    const int g = g0 + lane, e = g - front;
    int64_t lo = 0, hi = 0;
    if (g < count) {
      if (e < 0) {
        hi = clamp64(p.offsets[0], 0, p.total_rows);
      } else if (e >= p.groups) {
        lo = clamp64(p.offsets[p.groups], 0, p.total_rows);
        hi = p.total_rows;
      } else {
        expert_rows(p, e, lo, hi);
      }
    }
    const int64_t tiles = (hi - lo + BM - 1) / BM;
    int64_t incl = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t up = __shfl_up(incl, o);
      if (lane >= o) incl += up;
    }
    const int64_t sum = __shfl(incl, 63);
    if (mt < before + sum) {
      const unsigned long long over = __ballot(before + incl > mt);
      const int src = __ffsll(over) - 1;
      const int64_t first = __shfl(before + incl - tiles, src);
      const int64_t glo = __shfl(lo, src);
      row_end = __shfl(hi, src);
      row0 = glo + (mt - first) * BM;
      const int ge = g0 + src - front;
      expert = ge >= 0 && ge < p.groups ? ge : -1;
      return true;
    }
    before += sum;
  }
  return false;
}

template <typename T>
struct Frag;
template <>
struct Frag<__bf16> {
  static constexpr int VEC = 8, BK = 64;
  __device__ static __forceinline__ void mma(floatx16& acc, u32x4 a, u32x4 b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  }
};
template <>
struct Frag<float> {
  static constexpr int VEC = 4, BK = 32;
  // lanes 0-31 and 32-63 hold neighbouring chunks of 4 k: MFMA p reduces over k = {p, 4 + p}
  __device__ static __forceinline__ void mma(floatx16& acc, u32x4 a, u32x4 b) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[p]), __uint_as_float(b[p]), acc,
                                                 0, 0, 0);
  }
};

// 16 bytes from any address of T's alignment, of which the first `valid` elements exist; the
// others read as zero and are not touched. (A whole chunk is one 16-byte load: this part loads
// from any address.)
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* p, int valid) {
  constexpr int VEC = Frag<T>::VEC;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (valid >= VEC) {
    __builtin_memcpy(&v, p, 16);
  } else if (valid > 0) {
    T e[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = i < valid ? p[i] : (T)0.f;
    __builtin_memcpy(&v, e, 16);
  }
  return v;
}

// Any sizes, pitches and alignment of both types: 128 x 128 tiles, four waves of 64 x 64, k-tiles
// of 128 bytes a row loaded into registers one tile ahead and stored to LDS as [row][k] (144-byte
// rows: 16 rows' 16-byte reads cover the 64 banks once), a k-major operand transposed on the way.
template <typename T, typename TO, int FORM>
__global__ __launch_bounds__(256) void k_grouped(GroupedArgs p) {
  using F = Frag<T>;
  constexpr int BM = 128, BN = 128, VEC = F::VEC, BK = F::BK;
  constexpr int PITCH = BK + VEC;                        // 144 bytes
  constexpr int NCH = 4;                                 // chunks per thread and operand
  __shared__ __align__(16) T As[BM * PITCH];
  __shared__ __align__(16) T Bs[BN * PITCH];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int expert = 0;
  int64_t row0 = 0, row_end = 0;
  int m_tile = 0, n0;
  int64_t red;              // length of the reduction
  const T* A;
  const T* B;
  int m_valid, n_valid;
  if constexpr (FORM == TN) {
    const int tm = (p.N + BM - 1) / BM, per = tm * p.tiles_n;
    expert = blockIdx.x / per;
    const int t = blockIdx.x % per;
    m_tile = t / p.tiles_n;
    n0 = (t % p.tiles_n) * BN;
    expert_rows(p, expert, row0, row_end);
    red = row_end - row0;
    A = static_cast<const T*>(p.A) + row0 * p.lda + m_tile * BM;
    B = static_cast<const T*>(p.B) + row0 * p.ldb + n0;
    m_valid = p.N - m_tile * BM;
    n_valid = p.K - n0;
  } else {
    if (!find_row_tile(p, BM, blockIdx.x / p.tiles_n, expert, row0, row_end)) return;
    n0 = (int)(blockIdx.x % p.tiles_n) * BN;
    red = expert < 0 ? 0 : p.K;
    A = static_cast<const T*>(p.A) + row0 * p.lda;
    B = static_cast<const T*>(p.B) + (expert < 0 ? 0 : expert) * p.sB +
        (FORM == NT ? n0 * p.ldb : (int64_t)n0);
    m_valid = (int)(row_end - row0 < BM ? row_end - row0 : BM);
    n_valid = p.N - n0;
  }

  // Chunk q of this thread of a k-contiguous operand: row, first k; of a k-major one: k-row,
  // first column (16 k-rows x 4 chunks per wave: 64-byte pieces of a row).
  u32x4 ra[NCH], rb[NCH];
  auto load = [&](const T* base, int64_t ld, bool kmajor, int valid, int64_t k0, u32x4* r) {
#pragma unroll
    for (int q = 0; q < NCH; ++q) {
      if (!kmajor) {
        const int c = tid + 256 * q, row = c >> 3, kk = (c & 7) * VEC;
        const int64_t left = red - k0 - kk;
        r[q] = load_chunk(base + row * ld + k0 + kk,
                          row < valid ? (int)(left < VEC ? left : VEC) : 0);
      } else {
        constexpr int KW = BK / 16;                     // waves' worth of k-rows
        const int u = q * 4 + wave;                     // 16 units of 16 k-rows x 4 chunks
        const int kr = (u % KW) * 16 + (lane & 15);
        const int col = ((u / KW) * 4 + (lane >> 4)) * VEC;
        const int left = valid - col;
        r[q] = load_chunk(base + (k0 + kr) * ld + col, k0 + kr < red ? (left < VEC ? left : VEC) : 0);
      }
    }
  };
  auto store = [&](T* dst, bool kmajor, const u32x4* r) {
#pragma unroll
    for (int q = 0; q < NCH; ++q) {
      if (!kmajor) {
        const int c = tid + 256 * q, row = c >> 3, kk = (c & 7) * VEC;
        *reinterpret_cast<u32x4*>(dst + row * PITCH + kk) = r[q];
      } else {
        constexpr int KW = BK / 16;
        const int u = q * 4 + wave;
        const int kr = (u % KW) * 16 + (lane & 15);
        const int col = ((u / KW) * 4 + (lane >> 4)) * VEC;
        T e[VEC];
        __builtin_memcpy(e, &r[q], 16);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dst[(col + i) * PITCH + kr] = e[i];
      }
    }
  };

  floatx16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  const int wm = wave >> 1, wn = wave & 1;
  if (red > 0) {
    load(A, p.lda, FORM == TN, m_valid, 0, ra);
    load(B, p.ldb, FORM != NT, n_valid, 0, rb);
  }
  for (int64_t k0 = 0; k0 < red; k0 += BK) {
    store(As, FORM == TN, ra);
    store(Bs, FORM != NT, rb);
    __syncthreads();
    if (k0 + BK < red) {
      load(A, p.lda, FORM == TN, m_valid, k0 + BK, ra);
      load(B, p.ldb, FORM != NT, n_valid, k0 + BK, rb);
    }
#pragma unroll
    for (int s = 0; s < BK / (2 * VEC); ++s) {
      u32x4 a[2], b[2];
      const int kk = (2 * s + (lane >> 5)) * VEC;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *reinterpret_cast<const u32x4*>(As + (wm * 64 + 32 * i + (lane & 31)) * PITCH + kk);
        b[i] = *reinterpret_cast<const u32x4*>(Bs + (wn * 64 + 32 * i + (lane & 31)) * PITCH + kk);
      }
      // the B tile feeds the MFMA's A input: each lane holds 4 consecutive columns of one row
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) F::mma(acc[i][j], b[j], a[i]);
    }
    __syncthreads();
  }

  // acc[i][j][4g + e] is row wm*64 + 32i + (lane & 31), column wn*64 + 32j + 8g + 4(lane >> 5) + e.
  const int64_t crow = FORM == TN ? (int64_t)m_tile * BM : row0;
  const int64_t cbase = FORM == TN ? expert * p.sC : 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = wm * 64 + 32 * i + (lane & 31);
    if (m >= m_valid) continue;
    TO* out = static_cast<TO*>(p.C) + cbase + (crow + m) * p.ldc + n0;
    const TO* add = static_cast<const TO*>(p.D) + cbase + (crow + m) * p.ldc + n0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = wn * 64 + 32 * j + 8 * g + 4 * (lane >> 5);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (n + e >= n_valid) continue;
          float v = acc[i][j][4 * g + e];
          if (FORM == TN && p.D) v += p.beta * (float)add[n + e];
          out[n + e] = (TO)v;
        }
      }
  }
}

template <typename T, typename TO, int FORM>
hipError_t launch_grouped(const GroupedArgs& a, int64_t blocks, hipStream_t s) {
  hipLaunchKernelGGL((k_grouped<T, TO, FORM>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

constexpr int kTile = 128;
int64_t tiles_up(int64_t x, int64_t t) { return (x + t - 1) / t; }

}  // namespace

int64_t grouped_blocks(const GroupedDesc& d) {
  if (d.weight_grad) return d.groups * tiles_up(d.n, kTile) * tiles_up(d.k, kTile);
  // every expert can end in a part tile, and so can the rows of no expert
  return (tiles_up(d.total_rows, kTile) + d.groups + 2) *
         tiles_up(d.transpose_w ? d.k : d.n, kTile);
}

size_t grouped_workspace(const GroupedDesc&) { return 0; }

const char* grouped_name(const GroupedDesc& d) {
  const bool f = d.store == Store::F32;
  if (d.weight_grad) return f ? "grouped_wgrad_f32" : "grouped_wgrad_bf16";
  if (d.transpose_w) return f ? "grouped_nn_f32" : "grouped_nn_bf16";
  return f ? "grouped_nt_f32" : "grouped_nt_bf16";
}

hipError_t grouped(const GroupedDesc& d, hipStream_t s) {
  const int64_t blocks = grouped_blocks(d);
  if (blocks < 1 || blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  GroupedArgs a;
  a.A = d.A; a.B = d.B; a.D = d.D; a.C = d.C;
  a.lda = d.lda;
  a.offsets = d.offsets;
  a.total_rows = d.total_rows;
  a.groups = (int)d.groups;
  a.fill_rest = d.fill_rest ? 1 : 0;
  a.beta = d.beta;
  a.sB = a.sC = d.n * d.k;
  if (d.weight_grad) {
    a.ldb = d.ldb;
    a.ldc = d.k;
    a.N = (int)d.n;
    a.K = (int)d.k;
    a.tiles_n = (int)tiles_up(d.k, kTile);
    if (d.store == Store::F32) return launch_grouped<float, float, TN>(a, blocks, s);
    if (d.out_store == Store::F32) return launch_grouped<__bf16, float, TN>(a, blocks, s);
    return launch_grouped<__bf16, __bf16, TN>(a, blocks, s);
  }
  a.ldb = d.k;
  a.ldc = d.ldc;
  a.N = (int)(d.transpose_w ? d.k : d.n);
  a.K = (int)(d.transpose_w ? d.n : d.k);
  a.tiles_n = (int)tiles_up(a.N, kTile);
  if (d.store == Store::F32)
    return d.transpose_w ? launch_grouped<float, float, NN>(a, blocks, s)
                         : launch_grouped<float, float, NT>(a, blocks, s);
  return d.transpose_w ? launch_grouped<__bf16, __bf16, NN>(a, blocks, s)
                       : launch_grouped<__bf16, __bf16, NT>(a, blocks, s);
}

}  // namespace mns
