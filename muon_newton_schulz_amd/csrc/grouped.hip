// Products grouped by expert: rows of one token matrix, sorted by expert, against that expert's
// own weight matrix, with group sizes that only the device knows.
//
//   forward          Y_e  = X_e W_e^T        (k_grouped<..., NT>)
//   input gradient   dX_e = dY_e W_e         (k_grouped<..., NN>)
//   weight gradient  G_e  = beta C_e + dY_e^T X_e, reduced over the expert's rows (TN)
//   layer            Z_e  = X_e W_e^T + b_e, Y = act(Z) + R        (NT with LayerArgs)
//   its input's      dX_e = (dY_e W_e) act'(Z_e) + R               (NN with LayerArgs)
//
// Expert e owns rows [offsets[e], offsets[e + 1]) of the token matrices. The offsets are read by
// the kernels only: no host copy, no synchronisation, so the calls can be captured. Every offset
// is clamped to [0, total_rows] and an end before its begin is an empty group, so wrong offsets
// give wrong results but never an access outside the buffers.
#include "activation.h"
#include "grouped_walk.h"
#include "lds_dma.h"
#include "mns_internal.h"
#include "row_vectors.h"

#include <algorithm>
#include <type_traits>

namespace mns {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

enum Form { NT = 0, NN = 1, TN = 2 };

// A product with a layer's epilogue: NT: Z = X W^T + bias, C = act(Z) + R, Z kept where it is given;
// NN: C = (dY W) act'(Z) + R. The forward and input-gradient kernels take either arguments.
struct LayerArgs : GroupedArgs {
  const void* bias;             // groups x N, or null
  const void* R;                // the rows of C, pitch ldr, or null
  void* Z;                      // the rows of C, pitch ldz: written (NT) or read (NN), or null
  int64_t ldr, ldz;
  int act;
  int parts, part_tiles;        // k_grouped_split: parts of the reduction, tiles that have room for them
};
template <typename Args>
constexpr bool kLayer = std::is_same_v<Args, LayerArgs>;

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

// Writes a wave's FM x FN fragments of 32 x 32 at rows m0, columns n0 of the tile whose first
// element is `origin`: acc[i][j][4g + e] is row 32 i + (lane & 31), column 32 j + 8 g + 4 (lane >> 5)
// + e. Four columns go out as one vector; with ADD, beta D is added, its vectors of one fragment
// row all loaded before the first store.
template <typename TO, int FM, int FN, bool ADD>
__device__ __forceinline__ void store_fragments(const GroupedArgs& p, const floatx16 (&acc)[FM][FN],
                                                int64_t origin, int m0, int n0, int m_valid,
                                                int n_valid) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));     // addresses computed here, not kept across a caller's loop
  const TO* D = static_cast<const TO*>(p.D);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + 32 * i + (lane & 31);
    if (m >= m_valid) continue;
    const int64_t row = origin + m * (int)p.ldc;
    TO* out = static_cast<TO*>(p.C) + row;
    float add[FN * 4][4] = {};
    if (ADD && D) {
#pragma unroll
      for (int q = 0; q < FN * 4; ++q) {
        const int n = n0 + 32 * (q / 4) + 8 * (q % 4) + 4 * (lane >> 5);
        TO t[4];
        if (n + 4 <= n_valid) {
          __builtin_memcpy(t, D + row + n, sizeof(t));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = n + e < n_valid ? D[row + n + e] : (TO)0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) add[q][e] = (float)t[e];
      }
    }
#pragma unroll
    for (int q = 0; q < FN * 4; ++q) {
      const int n = n0 + 32 * (q / 4) + 8 * (q % 4) + 4 * (lane >> 5);
      TO t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = acc[i][q / 4][4 * (q % 4) + e];
        if (ADD && D) v += p.beta * add[q][e];
        t[e] = (TO)v;
      }
      if (n + 4 <= n_valid) {
        __builtin_memcpy(out + n, t, sizeof(t));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < n_valid) out[n + e] = t[e];
      }
    }
  }
}

// ---- the epilogue of a layer ------------------------------------------------------------------

// Zeros over a tile of rows that belong to no expert (m_rows x n_cols of it, threads of one block).
template <typename T, int FORM>
__device__ __forceinline__ void zero_tile(const LayerArgs& p, int64_t row, int col, int m_rows,
                                          int n_cols) {
  for (int i = threadIdx.x; i < m_rows * n_cols; i += blockDim.x) {
    const int m = i / n_cols, n = col + i % n_cols;
    static_cast<T*>(p.C)[(row + m) * p.ldc + n] = (T)0.f;
    if (FORM == NT && p.Z) static_cast<T*>(p.Z)[(row + m) * p.ldz + n] = (T)0.f;
  }
}

// A wave's fragments go through 4 KB of LDS of its own, 32 rows x 32 columns or 16 x 64 of float32 at a
// time, so that a lane holds eight consecutive columns of a row: the addends and outputs then move as
// whole pieces of 16 bytes, 128-byte lines of bfloat16, and one copy of the activation's code serves
// all fragments of a row. Used by every grouped kernel but those of 256 x 256 tiles (layer_rows) and of few
// rows (k_grouped_rows, whose fragments lie four columns a lane as they are). Latency of the operands'
// loads is what it adds (1021 rows, 5 experts of 513 x 1277, silu, a residual: 20.3 us, the product alone
// 18.4), so they are loaded a step ahead (without: 2 us more). Everything is float32 until the output's one
// rounding; act sees the sum, not Z as it is kept (the gradient then is that of the rounded Z, up to 2^-8 of it
// away).
//
// The epilogue of a wave's FM x FN fragments (as in store_fragments) at rows m0, columns n0 of the tile
// that starts at row `row`, column `col`, in FM * FN steps. load() takes a step's operands; a step's are
// loaded before the one before it is finished, the first ones by the caller where its registers allow
// that before the product itself.
template <typename T, int FORM, int FM, int FN>
struct Finish {
  static constexpr bool EXACT = sizeof(T) == 4;
  static constexpr int ROWS = 32 / FN, CH = 8 * FN, LANES = 4 * FN, STEP = 64 / LANES;
  struct Operands {
    Eight<T> z[2], r[2];
  };
  int ln, c, r0, n, left, col, m0, m_valid, expert;
  int64_t row;
  Eight<T> bias;
  Operands first;

  __device__ __forceinline__ Finish(int expert_, int64_t row_, int col_, int m0_, int n0,
                                    int m_valid_, int n_valid) {
    ln = threadIdx.x & 63;
    asm volatile("" : "+v"(ln));       // addresses computed here, not kept across a caller's loop
    c = ln % LANES;
    r0 = ln / LANES;
    n = n0 + 8 * c;
    left = n_valid - n;
    col = col_;
    m0 = m0_;
    m_valid = m_valid_;
    expert = expert_;
    row = row_;
  }
  // chunk k of staged row r: the 16-byte accesses of 16 lanes cover all banks, writing and reading
  __device__ __forceinline__ static int at(int r, int k) {
    return r * CH + (k ^ (FN == 2 ? r & 15 : (r >> 1) & 7));
  }
  __device__ __forceinline__ int row_of(int step) const {
    return m0 + 32 * (step / FN) + ROWS * (step % FN) + r0;
  }
  __device__ __forceinline__ void load(const LayerArgs& p, int step, Operands& o) const {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int m = row_of(step) + STEP * q, have = m < m_valid ? left : 0;
      if (FORM == NN)
        o.z[q].load(static_cast<const T*>(p.Z) + (row + m) * p.ldz + col + n, p.Z ? have : 0,
                    rows_end(static_cast<const T*>(p.Z), p, p.ldz, p.N));
      o.r[q].load(static_cast<const T*>(p.R) + (row + m) * p.ldr + col + n, p.R ? have : 0,
                  rows_end(static_cast<const T*>(p.R), p, p.ldr, p.N));
    }
  }
  __device__ __forceinline__ void load_first(const LayerArgs& p) {
    if (FORM == NT)
      bias.load(static_cast<const T*>(p.bias) + (int64_t)expert * p.N + col + n, p.bias ? left : 0,
                static_cast<const T*>(p.bias) + (int64_t)p.groups * p.N);
    load(p, 0, first);
  }
  __device__ __forceinline__ void run(const LayerArgs& p, const floatx16 (&acc)[FM][FN],
                                      floatx4* stage) const {
    Operands now = first;
#pragma unroll
    for (int step = 0; step < FM * FN; ++step) {
      const int i = step / FN, pass = step % FN;
      Operands next;
      if (step + 1 < FM * FN) load(p, step + 1, next);
      if (FN == 1 || ((ln >> 4) & 1) == pass) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            floatx4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e];
            stage[at(ln & (ROWS - 1), 8 * j + 2 * g + (ln >> 5))] = v;
          }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const floatx4 lo = stage[at(r0 + STEP * q, 2 * c)], hi = stage[at(r0 + STEP * q, 2 * c + 1)];
        const int m = row_of(step) + STEP * q;
        if (m >= m_valid || left <= 0) continue;
        float v[8], x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
        Eight<T> out;
        if constexpr (FORM == NT) {
          bias.get(x);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += x[e];
          if (p.Z) {
            out.set(v);
            out.store(static_cast<T*>(p.Z) + (row + m) * p.ldz + col + n, left);
          }
          activate<EXACT>(p.act, v);
        } else {
          now.z[q].get(x);
          times_slope<EXACT>(p.act, v, x);
        }
        now.r[q].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += x[e];
        out.set(v);
        out.store(static_cast<T*>(p.C) + (row + m) * p.ldc + col + n, left);
      }
      if (step + 1 < FM * FN) now = next;
    }
  }
};

// (a plain product has none)
struct NoFinish {
  template <typename... A>
  __device__ __forceinline__ NoFinish(A...) {}
};
template <typename Args, typename T, int FORM, int FM, int FN>
using FinishOf = std::conditional_t<kLayer<Args>, Finish<T, FORM, FM, FN>, NoFinish>;

// The other orientation (A feeds the MFMA's A input): element e of a lane is row m0 + 8 (e / 4)
// + 4 (lane >> 5) + e % 4, column n0 + (lane & 31). 32 lanes hold 32 neighbouring columns, so a
// float32 output and its addend move as whole 128-byte lines, straight from registers; bfloat16
// neighbours are paired (the even lane takes row e, the odd one row e + 1), 64 bytes of four rows
// a store. One fragment's addends, and its store:
template <typename TO>
__device__ __forceinline__ void load_addend(const GroupedArgs& p, int64_t origin, int m0, int n0,
                                            int m_valid, int n_valid, float (&add)[16]) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));     // addresses computed here, not kept across a caller's loop
  const TO* D = static_cast<const TO*>(p.D) + origin;
  const int n = n0 + (lane & 31);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int m = m0 + 8 * (e / 4) + 4 * (lane >> 5) + e % 4;
    // past the end: the tile's first element, in bounds and not used
    add[e] = (float)D[m < m_valid && n < n_valid ? m * (int)p.ldc + n : 0];
  }
}
template <typename TO>
__device__ __forceinline__ void store_lanes(const GroupedArgs& p, const floatx16& acc,
                                            int64_t origin, int m0, int n0, int m_valid,
                                            int n_valid, const float (&add)[16]) {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  TO* C = static_cast<TO*>(p.C) + origin;
  const int n = n0 + (lane & 31);
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const int m = m0 + 8 * (e / 4) + 4 * (lane >> 5) + e % 4;
    float v[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      v[r] = acc[e + r];
      if (p.D) v[r] += p.beta * add[e + r];
    }
    if constexpr (sizeof(TO) == 4) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (m + r < m_valid && n < n_valid) C[(m + r) * (int)p.ldc + n] = v[r];
    } else {
      const bool odd = lane & 1;
      const unsigned give = __builtin_bit_cast(unsigned, odd ? v[0] : v[1]);
      // quad_perm [1, 0, 3, 2]: the neighbour's value of the row this lane stores
      const float got = __builtin_bit_cast(
          float, __builtin_amdgcn_update_dpp(0u, give, 0xB1, 0xF, 0xF, true));
      const TO pair[2] = {(TO)(odd ? got : v[0]), (TO)(odd ? v[1] : got)};
      const int mm = m + odd, nn = n - odd;
      if (mm >= m_valid) continue;
      TO* dst = C + mm * (int)p.ldc + nn;
      if (nn + 1 < n_valid) __builtin_memcpy(dst, pair, sizeof(pair));
      else if (nn < n_valid) dst[0] = pair[0];
    }
  }
}

// A k-major bfloat16 W whose rows do not all start on 4 bytes (an odd pitch: every other one) is read from
// the element before, where that makes it so: loads between dwords take up to twice as long (input gradient,
// 16384 rows over 8 experts of 2048 x 4097: 999 -> 653 us; 1021 over 5 of 513 x 1277: 22.4 -> 18.4; where all
// rows start on 4 bytes it would cost 5 to 15 %, so the host chooses, FIX). As the elements go to LDS one by one, transposed, a
// chunk read one column early is stored one column early; column -1 has a place of its own in front, and
// the tile's last column is an element more a row.
template <bool FIX, typename T>
__device__ __forceinline__ int early(const T* at, const T* start) {
  return FIX && (reinterpret_cast<uintptr_t>(at) & 2) && at > start ? 1 : 0;
}

// Any sizes, pitches and alignment of both types: 128 x 128 tiles, four waves of 64 x 64, k-tiles
// of 128 bytes a row loaded into registers one tile ahead and stored to LDS as [row][k] (144-byte
// rows: 16 rows' 16-byte reads cover the 64 banks once), a k-major operand transposed on the way.
// With an addend, few rows: bound by HBM (384 rows over 16 experts of 2048 x 2048, float32 output: 105 us,
// 5.1 TB/s); else by the loads' latency (one k-tile ahead is what two blocks a CU have registers
// for; two ahead measured 10 to 60 % slower).
template <typename T, typename TO, int FORM, typename Args, bool FIX>
__global__ __launch_bounds__(256) void k_grouped(Args p) {
  using F = Frag<T>;
  constexpr int BM = 128, BN = 128, VEC = F::VEC, BK = F::BK;
  constexpr int PITCH = BK + VEC;                        // 144 bytes
  constexpr int NCH = 4;                                 // chunks per thread and operand
  __shared__ __align__(16) T As[BM * PITCH];
  __shared__ __align__(16) T Bbuf[(BN + (FIX ? 1 : 0)) * PITCH];
  T* const Bs = Bbuf + (FIX ? PITCH : 0);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int expert, lo, hi, m0, n0;
  int red;                  // length of the reduction
  const T* A;
  const T* B;
  const T* a_end = rows_end(static_cast<const T*>(p.A), p, p.lda, FORM == TN ? p.N : p.K);
  const T* b_end = FORM == TN ? rows_end(static_cast<const T*>(p.B), p, p.ldb, p.K)
                              : static_cast<const T*>(p.B) + p.groups * p.sB;
  int m_valid;
  if constexpr (FORM == TN) {
    const int per = (p.N + BM - 1) / BM * p.tiles_n, t = block_place() % per;
    expert = block_place() / per;
    if (expert >= p.groups) return;
    m0 = t / p.tiles_n * BM;
    n0 = t % p.tiles_n * BN;
    expert_rows(p, expert, lo, hi);
    red = hi - lo;
    A = static_cast<const T*>(p.A) + lo * p.lda + m0;
    B = static_cast<const T*>(p.B) + lo * p.ldb + n0;
    m_valid = p.N - m0;
  } else {
    Place at;
    if (!find_place(p, BM, p.tiles_n, p.fill_rest, walk_start(p, BM, p.tiles_n, p.fill_rest),
                    block_place(), at))
      return;
    expert = at.expert;
    m0 = at.lo + at.inside / p.tiles_n * BM;
    n0 = at.inside % p.tiles_n * BN;
    if constexpr (kLayer<Args>) {
      if (expert < 0) {
        zero_tile<T, FORM>(p, m0, n0, at.hi - m0 < BM ? at.hi - m0 : BM, p.N - n0 < BN ? p.N - n0 : BN);
        return;
      }
    }
    red = expert < 0 ? 0 : p.K;
    A = static_cast<const T*>(p.A) + m0 * p.lda;
    B = static_cast<const T*>(p.B) + (expert < 0 ? 0 : expert) * p.sB +
        (FORM == NT ? n0 * p.ldb : (int64_t)n0);
    m_valid = at.hi - m0;
  }
  const int n_valid = (FORM == TN ? p.K : p.N) - n0;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t origin = (FORM == TN ? expert * p.sC : 0) + m0 * p.ldc + n0;
  // The addend first: with few rows its bytes and the output's are what the call takes.
  float add[2][2][16];
  if (FORM == TN && p.D) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        load_addend<TO>(p, origin, wm * 64 + 32 * i, wn * 64 + 32 * j, m_valid, n_valid, add[i][j]);
  }

  // Chunk q of this thread of a k-contiguous operand: row, first k; of a k-major one: k-row,
  // first column (16 k-rows x 4 chunks per wave: 64-byte pieces of a row).
  u32x4 ra[NCH], rb[NCH];
  // Past the ends: rows of the reduction are zeros, and so are the reduction's columns (store); columns
  // of the output hold what follows in the operand and are not stored.
  auto load = [&](const T* base, int64_t ld, bool kmajor, int valid, int k0, const T* end, u32x4* r) {
#pragma unroll
    for (int q = 0; q < NCH; ++q) {
      if (!kmajor) {
        const int c = tid + 256 * q, row = c >> 3, kk = (c & 7) * VEC;
        const int left = red - k0 - kk;
        r[q] = load_piece_of_row(base + row * ld + k0 + kk, row < valid ? left : 0, end);
      } else {
        constexpr int KW = BK / 16;                     // waves' worth of k-rows
        const int u = q * 4 + wave;                     // 16 units of 16 k-rows x 4 chunks
        const int kr = (u % KW) * 16 + (lane & 15);
        const int col = ((u / KW) * 4 + (lane >> 4)) * VEC;
        const T* at = base + (int64_t)(k0 + kr) * ld + col;
        const int s = early<FIX>(at, static_cast<const T*>(p.B));
        const int left = valid - col + s;
        r[q] = load_piece_of_row(at - s, k0 + kr < red ? left : 0, end);
      }
    }
  };
  const T* last_at = B + (int64_t)tid * p.ldb + BN - 1;  // FIX: the last column of k-row tid
  auto last_missing = [&](int k0) {
    return tid < BK && early<FIX>(last_at + (int64_t)k0 * p.ldb - (BN - 1), (const T*)nullptr);
  };
  auto load_last = [&](int k0) {
    return last_missing(k0) && k0 + tid < red && n_valid >= BN ? last_at[(int64_t)k0 * p.ldb] : (T)0.f;
  };
  auto store_last = [&](int k0, T last) {
    if (last_missing(k0)) Bs[(BN - 1) * PITCH + tid] = last;
  };
  auto store = [&](T* dst, bool kmajor, int k0, const u32x4* r) {
#pragma unroll
    for (int q = 0; q < NCH; ++q) {
      if (!kmajor) {
        const int c = tid + 256 * q, row = c >> 3, kk = (c & 7) * VEC;
        *reinterpret_cast<u32x4*>(dst + row * PITCH + kk) =
            k0 + BK <= red ? r[q] : cut_chunk<T>(r[q], red - k0 - kk);
      } else {
        constexpr int KW = BK / 16;
        const int u = q * 4 + wave;
        const int kr = (u % KW) * 16 + (lane & 15);
        const int col = ((u / KW) * 4 + (lane >> 4)) * VEC;
        T e[VEC];
        __builtin_memcpy(e, &r[q], 16);
        T* at = dst + col * PITCH + kr;
        if (FIX) at -= early<FIX>(B + (int64_t)(k0 + kr) * p.ldb + col, static_cast<const T*>(p.B)) * PITCH;
#pragma unroll
        for (int i = 0; i < VEC; ++i) at[i * PITCH] = e[i];
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
  T last = (T)0.f;
  if (red > 0) {
    load(A, p.lda, FORM == TN, m_valid, 0, a_end, ra);
    load(B, p.ldb, FORM != NT, n_valid, 0, b_end, rb);
    if (FIX) last = load_last(0);
  }
  for (int k0 = 0; k0 < red; k0 += BK) {
    store(As, FORM == TN, k0, ra);
    store(Bs, FORM != NT, k0, rb);
    if (FIX) store_last(k0, last);
    __syncthreads();
    if (k0 + BK < red) {
      load(A, p.lda, FORM == TN, m_valid, k0 + BK, a_end, ra);
      load(B, p.ldb, FORM != NT, n_valid, k0 + BK, b_end, rb);
      if (FIX) last = load_last(k0 + BK);
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
      // B as the MFMA's A input: each lane holds 4 consecutive columns of one row; the other way
      // round, for the weight gradient: one column of 16 rows
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (FORM == TN) F::mma(acc[i][j], a[i], b[j]);
          else F::mma(acc[i][j], b[j], a[i]);
        }
    }
    __syncthreads();
  }

  if constexpr (FORM == TN) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        store_lanes<TO>(p, acc[i][j], origin, wm * 64 + 32 * i, wn * 64 + 32 * j, m_valid, n_valid,
                        add[i][j]);
  } else if constexpr (kLayer<Args>) {
    // (behind the loop's last barrier the operands' LDS is free)
    Finish<T, FORM, 2, 2> end(expert, m0, n0, wm * 64, wn * 64, m_valid, n_valid);
    end.load_first(p);
    end.run(p, acc, reinterpret_cast<floatx4*>(As) + wave * 256);
  } else {
    store_fragments<TO, 2, 2, false>(p, acc, origin, wm * 64, wn * 64, m_valid, n_valid);
  }
}

// The same for forwards and input gradients whose grid would leave CUs without work: 64 x 64 tiles,
// whose four waves split the reduction (wave w takes k-tiles w, w + 4, ...), each with its own LDS and
// no barrier in the loop; the four sums are added in wave order through LDS. A fourth of the steps
// of memory latency one after the other, and four times the blocks. Bound by those steps (1021 rows
// over 5 experts of 513 x 1277, bfloat16, input gradient: 18 us).
//
// A layer's reduction that is still long for its few tiles is cut into `parts` more (split_parts), a block
// each: their float32 sums go to p.partial and are added in part order by k_split_join (float32 input
// gradient of 141 rows over 2 experts of 6080 x 320: 162 -> 27 us, a call's 12 among them).

// A block's tile: false where there is none. part: of the reduction; slot: of p.partial's tiles (those
// of no expert have none), always below part_tiles where the offsets do not overlap.
template <typename Args>
__device__ __forceinline__ bool split_place(const Args& p, int lin, Place& at, int& slot) {
  constexpr int BM = 64;
  if (!find_place(p, BM, p.tiles_n, p.fill_rest, walk_start(p, BM, p.tiles_n, p.fill_rest), lin, at))
    return false;
  slot = lin;
  if constexpr (kLayer<Args>) {
    if (p.fill_rest)
      slot -= (clamp_row(p.offsets[0], 0, p.total_rows) + BM - 1) / BM * p.tiles_n;
    return p.parts == 1 || at.expert < 0 || (slot >= 0 && slot < p.part_tiles);
  }
  return true;
}

template <typename T, int FORM, typename Args, bool FIX>
__global__ __launch_bounds__(256) void k_grouped_split(Args p) {
  using F = Frag<T>;
  constexpr int BM = 64, BN = 64, VEC = F::VEC, BK = F::BK, PITCH = BK + VEC;
  constexpr int NCH = 8;                                 // chunks per lane and operand
  constexpr int WAVE = (BM + BN + (FIX ? 1 : 0)) * PITCH;   // elements of one wave's LDS
  __shared__ __align__(16) T lds[4 * WAVE];
  static_assert(sizeof(lds) >= 4 * 4 * 16 * 64 * sizeof(float), "the waves' sums fit");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Place at;
  int slot, part = 0;
  int lin = block_place();
  if constexpr (kLayer<Args>) {
    part = lin % p.parts;
    lin /= p.parts;
  }
  if (!split_place(p, lin, at, slot)) return;
  const int m0 = at.lo + at.inside / p.tiles_n * BM, n0 = at.inside % p.tiles_n * BN;
  const int m_valid = at.hi - m0, n_valid = p.N - n0;
  if constexpr (kLayer<Args>) {
    if (at.expert < 0) {
      if (part == 0)
        zero_tile<T, FORM>(p, m0, n0, m_valid < BM ? m_valid : BM, n_valid < BN ? n_valid : BN);
      return;
    }
  }
  const int red = at.expert < 0 ? 0 : p.K;
  int k_first = 0, k_end = red;                          // of this block's part, whole k-tiles
  if constexpr (kLayer<Args>) {
    const int tiles = (red + BK - 1) / BK;
    k_first = tiles * part / p.parts * BK;
    if (part + 1 < p.parts) k_end = tiles * (part + 1) / p.parts * BK;
  }
  const T* A = static_cast<const T*>(p.A) + m0 * p.lda;
  const T* B = static_cast<const T*>(p.B) + (at.expert < 0 ? 0 : at.expert) * p.sB +
               (FORM == NT ? n0 * p.ldb : (int64_t)n0);

  const T* a_end = rows_end(static_cast<const T*>(p.A), p, p.lda, p.K);
  const T* b_end = static_cast<const T*>(p.B) + p.groups * p.sB;
  auto load = [&](const T* base, int64_t ld, bool kmajor, int valid, int k0, const T* end, u32x4* r) {
#pragma unroll
    for (int q = 0; q < NCH; ++q) {
      if (!kmajor) {
        const int c = lane + 64 * q, row = c >> 3, kk = (c & 7) * VEC;
        r[q] = load_piece_of_row(base + row * ld + k0 + kk, row < valid ? red - k0 - kk : 0, end);
      } else {
        constexpr int KW = BK / 16;
        const int kr = (q % KW) * 16 + (lane & 15), col = ((q / KW) * 4 + (lane >> 4)) * VEC;
        const T* at = base + (int64_t)(k0 + kr) * ld + col;
        const int s = early<FIX>(at, static_cast<const T*>(p.B));
        r[q] = load_piece_of_row(at - s, k0 + kr < red ? valid - col + s : 0, end);
      }
    }
  };
  const T* last_at = B + (int64_t)lane * p.ldb + BN - 1; // FIX: the last column of k-row `lane`
  auto last_missing = [&](int k0) {
    return early<FIX>(last_at + (int64_t)k0 * p.ldb - (BN - 1), (const T*)nullptr);
  };
  auto load_last = [&](int k0) {
    return last_missing(k0) && k0 + lane < red && n_valid >= BN ? last_at[(int64_t)k0 * p.ldb] : (T)0.f;
  };
  auto store_last = [&](T* dst, int k0, T last) {
    if (last_missing(k0)) dst[(BN - 1) * PITCH + lane] = last;
  };
  auto store = [&](T* dst, bool kmajor, int k0, const u32x4* r) {
#pragma unroll
    for (int q = 0; q < NCH; ++q) {
      if (!kmajor) {
        const int c = lane + 64 * q, row = c >> 3, kk = (c & 7) * VEC;
        *reinterpret_cast<u32x4*>(dst + row * PITCH + kk) =
            k0 + BK <= red ? r[q] : cut_chunk<T>(r[q], red - k0 - kk);
      } else {
        constexpr int KW = BK / 16;
        const int kr = (q % KW) * 16 + (lane & 15), col = ((q / KW) * 4 + (lane >> 4)) * VEC;
        T e[VEC];
        __builtin_memcpy(e, &r[q], 16);
        T* at = dst + col * PITCH + kr;
        if (FIX) at -= early<FIX>(B + (int64_t)(k0 + kr) * p.ldb + col, static_cast<const T*>(p.B)) * PITCH;
#pragma unroll
        for (int i = 0; i < VEC; ++i) at[i * PITCH] = e[i];
      }
    }
  };
  static_assert(!FIX || BK == 64, "a lane for each k-row");
  // wave w finishes fragment (w / 2, w % 2)
  const int mi = 32 * (wave >> 1), nj = 32 * (wave & 1);
  FinishOf<Args, T, FORM, 1, 1> end(at.expert, m0, n0, mi, nj, m_valid, n_valid);
  if constexpr (kLayer<Args>) {
    if (p.parts == 1) end.load_first(p);
  }
  const bool two = m_valid > 32;                         // else the rows behind are not multiplied
  floatx16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  T* As = lds + wave * WAVE;
  T* Bs = As + (BM + (FIX ? 1 : 0)) * PITCH;
  u32x4 ra[NCH], rb[NCH];
  T last = (T)0.f;
  int k0 = k_first + wave * BK;
  if (k0 < k_end) {
    load(A, p.lda, false, m_valid, k0, a_end, ra);
    load(B, p.ldb, FORM != NT, n_valid, k0, b_end, rb);
    if (FIX) last = load_last(k0);
  }
  for (; k0 < k_end; k0 += 4 * BK) {
    store(As, false, k0, ra);
    store(Bs, FORM != NT, k0, rb);
    if (FIX) store_last(Bs, k0, last);
    if (k0 + 4 * BK < k_end) {
      load(A, p.lda, false, m_valid, k0 + 4 * BK, a_end, ra);
      load(B, p.ldb, FORM != NT, n_valid, k0 + 4 * BK, b_end, rb);
      if (FIX) last = load_last(k0 + 4 * BK);
    }
#pragma unroll
    for (int s = 0; s < BK / (2 * VEC); ++s) {
      u32x4 a[2], b[2];
      const int kk = (2 * s + (lane >> 5)) * VEC;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *reinterpret_cast<const u32x4*>(As + (32 * i + (lane & 31)) * PITCH + kk);
        b[i] = *reinterpret_cast<const u32x4*>(Bs + (32 * i + (lane & 31)) * PITCH + kk);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i == 0 || two) {
#pragma unroll
          for (int j = 0; j < 2; ++j) F::mma(acc[i][j], b[j], a[i]);
        }
    }
  }
  __syncthreads();
  float(*sums)[4][16][64] = reinterpret_cast<float(*)[4][16][64]>(lds);     // [wave][fragment]
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int e = 0; e < 16; ++e) sums[wave][f][e][lane] = acc[f >> 1][f & 1][e];
  __syncthreads();
  floatx16 sum[1][1];
#pragma unroll
  for (int e = 0; e < 16; ++e)
    sum[0][0][e] = sums[0][wave][e][lane] + sums[1][wave][e][lane] + sums[2][wave][e][lane] +
                   sums[3][wave][e][lane];
  if constexpr (kLayer<Args>) {
    if (p.parts > 1) {
      if (mi >= m_valid || nj >= n_valid) return;        // a fragment without an element
      float* out = p.partial + ((((int64_t)slot * p.parts + part) * 4 + wave) * 64 + lane) * 16;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        floatx4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = sum[0][0][4 * g + e];
        reinterpret_cast<floatx4*>(out)[g] = v;
      }
      return;
    }
    __syncthreads();                   // every wave has read the sums
    end.run(p, sum, reinterpret_cast<floatx4*>(lds) + wave * 256);
  } else {
    store_fragments<T, 1, 1, false>(p, sum, m0 * p.ldc + n0, mi, nj, m_valid, n_valid);
  }
}

// Adds a tile's parts in part order and finishes the layer: one block a tile, one fragment a wave.
template <typename T, int FORM>
__global__ __launch_bounds__(256) void k_split_join(LayerArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Place at;
  int slot;
  if (!split_place(p, block_place(), at, slot) || at.expert < 0) return;
  const int m0 = at.lo + at.inside / p.tiles_n * 64, n0 = at.inside % p.tiles_n * 64;
  const int m_valid = at.hi - m0, n_valid = p.N - n0;
  const int mi = 32 * (wave >> 1), nj = 32 * (wave & 1);
  if (mi >= m_valid || nj >= n_valid) return;
  Finish<T, FORM, 1, 1> end(at.expert, m0, n0, mi, nj, m_valid, n_valid);
  end.load_first(p);
  floatx16 sum[1][1];
#pragma unroll
  for (int e = 0; e < 16; ++e) sum[0][0][e] = 0.f;
  const floatx4* src =
      reinterpret_cast<const floatx4*>(p.partial) + (((int64_t)slot * p.parts * 4 + wave) * 64 + lane) * 4;
#pragma unroll 4
  for (int part = 0; part < p.parts; ++part) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const floatx4 v = src[part * 1024 + g];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[0][0][4 * g + e] += v[e];
    }
  }
  __shared__ floatx4 stage[4 * 256];
  end.run(p, sum, stage + wave * 256);
}

// Few rows per expert (forward): the product is bound by reading the weights once, so the weights
// go straight from memory into MFMA operands, 64 bytes of 16 rows per load, with nothing staged
// and no barrier in the loop; the tokens of the row tile (16 MT rows) are read the same way and
// come from the caches. A wave owns 16 NT weight rows. WK = 4: the block's four waves split the
// reduction and add their sums through LDS in wave order (more waves in flight where there are
// few weight rows); WK = 1: they own 16 NT rows each.
//
// A 16-byte chunk per lane holds consecutive k of one row for both operands, so any k order the
// MFMA uses inside a step is the same on both sides. Loads are D - 1 steps ahead. 12 rows each, 8
// experts of 4096 x 2048: 35 us, 3.8 TB/s of weights; 613 rows over 9 of 777 x 331, float32: 13 us, the
// latency of a launch and a few loads.
template <typename T>
struct Small;
template <>
struct Small<__bf16> {
  __device__ static __forceinline__ void mma(floatx4& acc, u32x4 a, u32x4 b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  }
};
template <>
struct Small<float> {
  __device__ static __forceinline__ void mma(floatx4& acc, u32x4 a, u32x4 b) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[p]), __uint_as_float(b[p]), acc,
                                                 0, 0, 0);
  }
};

template <typename T, int MT, int NTW, int WK, typename Args>
__global__ __launch_bounds__(256) void k_grouped_rows(Args p) {
  constexpr int VEC = Frag<T>::VEC, STEP = 4 * VEC;     // k per step: 64 bytes of a row
  constexpr int BM = 16 * MT, BN = 16 * NTW * (4 / WK);
  constexpr int D = MT >= 4 ? 3 : 4;                    // operand sets: loads D - 1 steps ahead
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Place at;
  if (!find_place(p, BM, p.tiles_n, p.fill_rest, walk_start(p, BM, p.tiles_n, p.fill_rest),
                    block_place(), at))
      return;
  const int expert = at.expert;
  const int row0 = at.lo + at.inside / p.tiles_n * BM;
  const int n0 = at.inside % p.tiles_n * BN + (WK == 1 ? wave * 16 * NTW : 0);
  const int m_valid = at.hi - row0 < BM ? at.hi - row0 : BM;
  if constexpr (kLayer<Args>) {
    if (expert < 0) {
      const int col = at.inside % p.tiles_n * BN;
      zero_tile<T, NT>(p, row0, col, m_valid, p.N - col < BN ? p.N - col : BN);
      return;
    }
  }
  const int K = expert < 0 ? 0 : p.K;
  const int steps = (K + STEP - 1) / STEP;
  const int s_begin = WK == 1 ? 0 : (int)((int64_t)wave * steps / WK);
  const int s_end = WK == 1 ? steps : (int)((int64_t)(wave + 1) * steps / WK);
  const int whole = K / STEP;                           // steps without a tail

  // Rows past the tile's last one (and weight rows past N) read the last one again; their
  // products are not stored.
  const int r16 = lane & 15, kc = (lane >> 4) * VEC;
  const T* xp[MT];
  const T* wp[NTW];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * i + r16;
    xp[i] = static_cast<const T*>(p.A) +
            (int64_t)(row0 + (m < m_valid ? m : m_valid - 1)) * p.lda + kc;
  }
#pragma unroll
  for (int j = 0; j < NTW; ++j) {
    const int n = n0 + 16 * j + r16;
    wp[j] = static_cast<const T*>(p.B) + (expert < 0 ? 0 : expert) * p.sB +
            (int64_t)(n < p.N ? n : p.N - 1) * p.ldb + kc;
  }
  floatx4 acc[MT][NTW];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NTW; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  // A layer's bias and residual at a fragment's place; where the waves share fragments, those of a wave's
  // first one are loaded before the product.
  T bias[4] = {}, res[4] = {};
  auto operands = [&](int i, int j) {
    if constexpr (kLayer<Args>) {
      const int m = 16 * i + r16, n = n0 + 16 * j + 4 * (lane >> 4);
      auto load = [&](const T* src, T (&t)[4]) {
        if (n + 4 <= p.N) {
          __builtin_memcpy(t, src, sizeof(t));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = n + e < p.N ? src[e] : (T)0.f;
        }
      };
      if (p.bias) load(static_cast<const T*>(p.bias) + (int64_t)expert * p.N + n, bias);
      if (p.R && m < m_valid) load(static_cast<const T*>(p.R) + (int64_t)(row0 + m) * p.ldr + n, res);
    }
  };
  if (WK > 1 && wave < MT * NTW) operands(wave / NTW, wave % NTW);

  u32x4 xa[D][MT], wa[D][NTW];
  auto load = [&](int s, int d) {
    const int64_t o = (int64_t)s * STEP;
#pragma unroll
    for (int j = 0; j < NTW; ++j) __builtin_memcpy(&wa[d][j], wp[j] + o, 16);
#pragma unroll
    for (int i = 0; i < MT; ++i) __builtin_memcpy(&xa[d][i], xp[i] + o, 16);
  };
  auto mul = [&](int d) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NTW; ++j) Small<T>::mma(acc[i][j], wa[d][j], xa[d][i]);
  };
  // Whole steps s_begin .. w_end - 1, step s in set (s - s_begin) % D. A load past the last one
  // reads the last step again (its set is not used), so the loop has no tests between loads.
  const int w_end = s_end < whole ? s_end : whole;
  if (w_end > s_begin) {
    const int last = w_end - 1;
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load(s_begin + d < last ? s_begin + d : last, d);
    int s = s_begin;
    for (; s + D <= w_end; s += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int ahead = s + d + D - 1;
        load(ahead < last ? ahead : last, (d + D - 1) % D);
        mul(d);
      }
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (s + d < w_end) mul(d);
  }
  for (int s = w_end > s_begin ? w_end : s_begin; s < s_end; ++s) {     // the step with the tail
    const int64_t o = (int64_t)s * STEP;
    const int left = K - s * STEP - kc;
    u32x4 w[NTW], x[MT];
#pragma unroll
    for (int j = 0; j < NTW; ++j)
      w[j] = load_piece_of_row(wp[j] + o, left, static_cast<const T*>(p.B) + p.groups * p.sB);
#pragma unroll
    for (int i = 0; i < MT; ++i)
      x[i] = load_piece_of_row(xp[i] + o, left, rows_end(static_cast<const T*>(p.A), p, p.lda, p.K));
#pragma unroll
    for (int j = 0; j < NTW; ++j) w[j] = cut_chunk<T>(w[j], left);
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = cut_chunk<T>(x[i], left);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NTW; ++j) Small<T>::mma(acc[i][j], w[j], x[i]);
  }

  // acc[i][j][e]: token 16 i + (lane & 15), weight row n0 + 16 j + 4 (lane >> 4) + e.
  auto put = [&](int i, int j, const floatx4& v) {
    const int m = 16 * i + r16, n = n0 + 16 * j + 4 * (lane >> 4);
    if (m >= m_valid) return;
    auto store = [&](void* base, int64_t ld, const float (&x)[4]) {
      T* out = static_cast<T*>(base) + (int64_t)(row0 + m) * ld + n;
      T t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = (T)x[e];
      if (n + 4 <= p.N) {
        __builtin_memcpy(out, t, sizeof(t));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) out[e] = t[e];
      }
    };
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = v[e];
    if constexpr (kLayer<Args>) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += (float)bias[e];
      if (p.Z) store(p.Z, p.ldz, x);
      activate<sizeof(T) == 4>(p.act, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += (float)res[e];
    }
    store(p.C, p.ldc, x);
  };
  if constexpr (WK == 1 && kLayer<Args>) {
    // a row of fragments at a time through LDS, so that the epilogue is one loop's body
    __shared__ floatx4 row[4][NTW][64];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int j = 0; j < NTW; ++j) row[wave][j][lane] = acc[i][j];
#pragma unroll 1
      for (int j = 0; j < NTW; ++j) {
        operands(i, j);
        put(i, j, row[wave][j][lane]);
      }
    }
  } else if constexpr (WK == 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NTW; ++j) put(i, j, acc[i][j]);
  } else if constexpr (kLayer<Args>) {
    __shared__ floatx4 ex[WK][MT * NTW][64];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NTW; ++j) ex[wave][i * NTW + j][lane] = acc[i][j];
    __syncthreads();
#pragma unroll 1
    for (int t = wave; t < MT * NTW; t += WK) {
      floatx4 v = ex[0][t][lane];
#pragma unroll
      for (int w = 1; w < WK; ++w) v += ex[w][t][lane];
      if (t != wave) operands(t / NTW, t % NTW);
      put(t / NTW, t % NTW, v);
    }
  } else {
    __shared__ floatx4 ex[WK][MT * NTW][64];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NTW; ++j) ex[wave][i * NTW + j][lane] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NTW; ++j) {
        const int t = i * NTW + j;
        if (t % WK != wave) continue;
        floatx4 v = ex[0][t][lane];
#pragma unroll
        for (int w = 1; w < WK; ++w) v += ex[w][t][lane];
        put(i, j, v);
      }
  }
}

// ---- large products, bfloat16 --------------------------------------------------------------
//
// 256 x 256 tiles, eight waves of 128 x 64 (2 x 4), k-tiles of 64 moved to LDS by DMA, double
// buffered: the main loop of the Newton-Schulz product (gemm.hip), for ragged rows and for both
// operands in either order. An operand whose rows run along the reduction lies in LDS as
// [row][k] in 16-byte chunks, chunk c of row r at c ^ ((r ^ (r >> 3 & 3)) & 7); one whose rows run
// along the output (W in dX = dY W, both in dY^T X) lies as [k][256 columns], chunk c of k-row r
// at c ^ 4 (r & 3), and is read through the transposing LDS load.
//
// Nothing is masked in the loop: an operand row past the end of its matrix lies past the buffer
// resource's end and reads as zero, and a row of the next expert only feeds output rows that are
// not stored. For the weight gradient the reduction ends inside a k-tile: the resources end at
// the expert's last row, so the rest of the tile is zeros for both operands; they start at the
// k-tile (not at the expert), so offsets stay below 2 GiB however many rows an expert has.

// Tile (tm, tn) of place `t` among tiles_m x tiles_n: groups of 4 row tiles, column by column inside a
// group, so that tiles in flight together share operand rows.
__device__ __forceinline__ void tile_order(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per = 4 * tiles_n, g = t / per, l = t % per;
  const int rest = tiles_m - 4 * g, size = rest < 4 ? rest : 4;
  tm = 4 * g + l % size;
  tn = l / size;
}

// Blocks go round the 8 XCDs (L2 domains) one by one: block b of a window of 256 takes the window's
// tile xcd_order(b), so the 32 CUs of an XCD work on 32 consecutive tiles, and an expert with many
// rows is spread over the XCDs.
__device__ __forceinline__ int xcd_order(int b) { return (b & 7) * 32 + (b >> 3); }

// How the tiles of a call are dealt to the 256 blocks: whole rounds first; a last round that would
// be at most half full is cut along the reduction into `split` parts a tile, whose float32 sums
// k_grouped_join adds in part order.
struct Deal {
  int rounds, tail, split;
};
__device__ __forceinline__ Deal deal(int total, int cap) {
  Deal d;
  d.rounds = total >> 8;
  d.tail = total & 255;
  int s = d.tail > 0 ? 256 / d.tail : 1;
  if (s > cap) s = cap;
  d.split = s < 1 ? 1 : s;
  return d;
}

// Weight gradients with at most 64 experts: experts with the most rows first (ties: in order), so
// that the blocks' last tiles are short ones. This lane's expert's rank.
__device__ __forceinline__ int rows_rank(const GroupedArgs& p) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = 0;
  if (lane < p.groups) expert_rows(p, lane, lo, hi);
  const int mine = hi - lo;
  int rank = 0;
  for (int l = 0; l < p.groups; ++l) {
    const int other = __builtin_amdgcn_readlane(mine, l);
    rank += other > mine || (other == mine && l < lane);
  }
  return lane < p.groups ? rank : -1;
}

// One tile (or a part of its reduction) in scalar registers: where its operands start and how many
// bytes behind that exist, its k-tiles, its output.
struct Unit {
  const char* A;
  const char* B;
  int64_t a_bytes, b_bytes;     // forward, input gradient
  int rows;                     // weight gradient: rows of the reduction
  int KL;
  int m_valid, n_valid;
  int64_t origin;
  int slot;                     // of the part's sums; -1: the whole tile
};
struct LayerUnit : Unit {
  int expert, row, col;         // of the tile
};

// The tile of position lin: expert, rows of the expert, tile coordinates in the output.
template <int FORM>
__device__ __forceinline__ bool tile_at(const GroupedArgs& p, const Walk& w, int rank, int lin,
                                        int& expert, int& lo, int& hi, int& m0, int& n0) {
  int tm, tn;
  if constexpr (FORM == TN) {
    const int tiles_m = (p.N + 255) / 256, per = tiles_m * p.tiles_n;
    if (lin >= w.total) return false;
    expert = lin / per;
    if (p.groups <= 64) expert = __ffsll((unsigned long long)__ballot(rank == expert)) - 1;
    tile_order(lin % per, tiles_m, p.tiles_n, tm, tn);
    expert_rows(p, expert, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    m0 = tm * 256;
  } else {
    Place at;
    if (!find_place(p, 256, p.tiles_n, 0, w, lin, at)) return false;
    expert = at.expert;
    lo = at.lo;
    hi = at.hi;
    tile_order(at.inside, (hi - lo + 255) / 256, p.tiles_n, tm, tn);
    m0 = lo + tm * 256;
  }
  n0 = tn * 256;
  return true;
}

// A block works through its units (every 256th tile, then at most one of the last round) without
// a break between them: the DMA runs two k-tiles ahead across the end of a tile, so the next
// tile's first k-tiles land while this one's last products and its epilogue run.
//
// 16384 rows over 32 experts of 8192 x 1024: forward 298 us, input gradient 310 with the join, weight
// gradient 334 (923, 887, 823 TFLOP/s; before the tiles ran into each other 329, 384, 442). The matrix
// units are busy 51, 51 and 42 % of the cycles, at 1.76 to 1.9 GHz (the power limit; 240 to 270 us before
// the clock comes down). The other half: part tiles (up to 255 rows of every expert's last one), an
// epilogue every 16 k-tiles (forward), 1.3 rounds of tiles (input gradient), the transposing reads'
// waits and 537 MB of output after eight k-tiles a tile (weight gradient). 16 rows over 32 experts: 46 us,
// the weights at 5.8 TB/s.
// (ACT, KEEP, RES: a layer's activation, whether Z is kept and whether there is a residual. As run-time
// choices their branches in the epilogue made the compiler spill up to 500 bytes a lane.)
template <typename TO, int FORM, bool ADD, typename Args, int ACT = ACT_NONE, bool KEEP = false,
          bool RES = false>
__global__ __launch_bounds__(512) void k_grouped_big(Args p) {
  constexpr int BM = 256, BN = 256, BK = 64, FM = 4, FN = 2, INST = 4;   // DMA per wave and operand
  constexpr int SLOT = 256 * kChunks;                   // u32x4 of one operand's k-tile (32 KB)
  constexpr bool AK = FORM == TN, BKM = FORM != NT;     // operand stored along the output
  constexpr int KROW = 512;                             // bytes of a [k][256] LDS row
  __shared__ u32x4 lds[5 * SLOT];                       // A: slots 0, 1; B: slots 2, 3, 4
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int block = xcd_order(blockIdx.x);

  Walk walk = {};
  int rank = -1;
  if constexpr (FORM == TN) {
    if (p.groups <= 64) rank = rows_rank(p);
    walk.total = (p.N + BM - 1) / BM * p.tiles_n * p.groups;
  } else {
    walk = walk_start(p, BM, p.tiles_n, 0);
  }
  const Deal dl = deal(walk.total, p.split_cap);

  using TileUnit = std::conditional_t<kLayer<Args>, LayerUnit, Unit>;
  auto unit = [&](int i, TileUnit& u) {
    int part = 0, parts = 1;
    int lin = i * 256 + block;
    u.slot = -1;
    if (i > dl.rounds) return false;
    if (i == dl.rounds) {                   // the last round, spread evenly over the XCDs
      const int units = dl.tail * dl.split, share = (units + 7) / 8;
      const int at = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
      if ((int)(blockIdx.x >> 3) >= share || at >= units) return false;
      part = at / dl.tail;
      parts = dl.split;
      if (parts > 1) u.slot = at;
      lin = i * 256 + at % dl.tail;
    }
    int expert, lo, hi, m0, n0;
    if (!tile_at<FORM>(p, walk, rank, lin, expert, lo, hi, m0, n0)) return false;
    const int red = FORM == TN ? hi - lo : p.K, tiles = (red + BK - 1) / BK;
    const int k0 = parts > 1 ? part * tiles / parts : 0;      // parts <= 16, tiles < 2^26
    const int k1 = parts > 1 ? (part + 1) * tiles / parts : tiles;
    u.KL = k1 - k0 < 2 ? 2 : k1 - k0;                   // the DMA looks two k-tiles ahead
    u.n_valid = (FORM == TN ? p.K : p.N) - n0;
    if constexpr (kLayer<Args>) {
      u.expert = expert;
      u.row = m0;
      u.col = n0;
    }
    if constexpr (FORM == TN) {
      const int left = red - k0 * BK, most = (k1 - k0) * BK;
      u.rows = left < most ? left : most;
      u.m_valid = p.N - m0;
      u.A = static_cast<const char*>(p.A) + ((lo + (int64_t)k0 * BK) * p.lda + m0) * 2;
      u.B = static_cast<const char*>(p.B) + ((lo + (int64_t)k0 * BK) * p.ldb + n0) * 2;
      u.a_bytes = u.b_bytes = 0;
      u.origin = expert * p.sC + m0 * p.ldc + n0;
    } else {
      u.rows = 0;
      u.m_valid = hi - m0;
      u.A = static_cast<const char*>(p.A) + (m0 * p.lda + k0 * BK) * 2;
      u.a_bytes = ((int64_t)(u.m_valid - 1) * p.lda + p.K - k0 * BK) * 2;
      const char* W = static_cast<const char*>(p.B) + expert * p.sB * 2;
      u.B = W + (BKM ? (int64_t)k0 * BK * p.ldb + n0 : n0 * p.ldb + k0 * BK) * 2;
      u.b_bytes = (BKM ? (int64_t)(p.K - k0 * BK) * p.ldb - n0
                       : (int64_t)(p.N - n0) * p.ldb - k0 * BK) * 2;
      u.origin = m0 * p.ldc + n0;
    }
    return true;
  };
  // Resource of k-tile kt of a unit: the unit's (k-tiles by offset), or, for the weight gradient, one
  // that starts at the k-tile and ends with the unit's last row.
  auto res = [&](const Unit& u, int kt, bool b) {
    if constexpr (FORM == TN) {
      const int64_t ld = b ? p.ldb : p.lda;
      const int64_t left = ((int64_t)(u.rows - kt * BK - 1) * ld + (b ? u.n_valid : u.m_valid)) * 2;
      return make_rsrc((b ? u.B : u.A) + kt * BK * ld * 2, u.rows > kt * BK ? left : 0);
    } else {
      return b ? make_rsrc(u.B, u.b_bytes) : make_rsrc(u.A, u.a_bytes);
    }
  };
  auto koff = [&](int kt, bool b) {
    if constexpr (FORM == TN) return 0;
    else return b && BKM ? kt * BK * (int)p.ldb * 2 : kt * BK * 2;
  };

  // Per-lane byte offsets of this wave's DMA instructions (see the layouts above).
  int offA[INST], offB[INST];
  auto lane_offset = [&](int i, bool kmajor, int64_t ld) {
    if (kmajor) {
      const int kr = 2 * (wave * INST + i) + (lane >> 5);
      return (kr * (int)ld + 8 * ((lane & 31) ^ (4 * (kr & 3)))) * 2;
    }
    const int row = (wave * INST + i) * 8 + (lane >> 3);
    return (row * (int)ld + 8 * ((lane & 7) ^ ((row ^ ((row >> 3) & 3)) & 7))) * 2;
  };
#pragma unroll
  for (int i = 0; i < INST; ++i) {
    offA[i] = lane_offset(i, AK, p.lda);
    offB[i] = lane_offset(i, BKM, p.ldb);
  }

  floatx16 acc[FM][FN];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  };

  const int arow = wm * 128 + (lane & 31), brow = wn * 64 + (lane & 31);
  u32x4 af[2][FM], bf[2][FN];
  // Transposing reads: in each 16-lane group G = lane / 16, lane 4s + a points at 8 bytes of k-row
  // 8 (G / 2) + s (+ 4 for the second read), columns c .. c + 3, c = first + 16 (G % 2) + 4 a, and
  // lane 4a + b receives the four k of column c + b: each lane ends with 8 consecutive k of its
  // row of the fragment, as the MFMA expects.
  uint32_t a_addr[FM], b_addr[FN];
  {
    const int G = lane >> 4, sq = (lane & 15) >> 2, a4 = lane & 3, kb = 8 * (G >> 1) + sq;
    const uint32_t base = lds_address(lds);
    auto address = [&](int first) {
      const int c = first + 16 * (G & 1) + 4 * a4;
      return (uint32_t)(kb * KROW + ((c >> 3) ^ (4 * (kb & 3))) * 16 + (c & 7) * 2);
    };
#pragma unroll
    for (int i = 0; i < FM; ++i) a_addr[i] = base + address(wm * 128 + 32 * i);
#pragma unroll
    for (int j = 0; j < FN; ++j) b_addr[j] = base + 2 * SLOT * 16 + address(wn * 64 + 32 * j);
  }
  auto load_frags = [&](int a, int b, int ks, int slot) {
    const int ch = 2 * ks + (lane >> 5);
    if constexpr (!AK) {
#pragma unroll
      for (int i = 0; i < FM; ++i) af[slot][i] = lds[a * SLOT + swz(arow + 32 * i, ch)];
    }
    if constexpr (!BKM) {
#pragma unroll
      for (int j = 0; j < FN; ++j) bf[slot][j] = lds[(2 + b) * SLOT + swz(brow + 32 * j, ch)];
    }
  };
  // The transposing loads wait for themselves (the compiler would wait for every outstanding DMA
  // first); outputs are early-clobber, and the fragments that the MFMAs before them read are
  // inputs, so none of those registers is written while an MFMA may still read it.
  auto load_tr = [&](int a, int b, int ks, int slot) {
    const uint32_t oa = (uint32_t)(a * SLOT * 16 + ks * 16 * KROW);
    const uint32_t ob = (uint32_t)(b * SLOT * 16 + ks * 16 * KROW);
    const int ps = slot ^ 1;
    u32x2 t0, t1, t2, t3, s0, s1, s2, s3, s4, s5, s6, s7;
    if constexpr (AK) {
      asm volatile(
          "ds_read_b64_tr_b16 %0, %12\n\t"
          "ds_read_b64_tr_b16 %1, %12 offset:2048\n\t"
          "ds_read_b64_tr_b16 %2, %13\n\t"
          "ds_read_b64_tr_b16 %3, %13 offset:2048\n\t"
          "ds_read_b64_tr_b16 %4, %14\n\t"
          "ds_read_b64_tr_b16 %5, %14 offset:2048\n\t"
          "ds_read_b64_tr_b16 %6, %15\n\t"
          "ds_read_b64_tr_b16 %7, %15 offset:2048\n\t"
          "ds_read_b64_tr_b16 %8, %16\n\t"
          "ds_read_b64_tr_b16 %9, %16 offset:2048\n\t"
          "ds_read_b64_tr_b16 %10, %17\n\t"
          "ds_read_b64_tr_b16 %11, %17 offset:2048\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(t0), "=&v"(t1), "=&v"(t2), "=&v"(t3), "=&v"(s0), "=&v"(s1), "=&v"(s2),
            "=&v"(s3), "=&v"(s4), "=&v"(s5), "=&v"(s6), "=&v"(s7)
          : "v"(b_addr[0] + ob), "v"(b_addr[1] + ob), "v"(a_addr[0] + oa), "v"(a_addr[1] + oa),
            "v"(a_addr[2] + oa), "v"(a_addr[3] + oa), "v"(af[ps][0]), "v"(af[ps][1]),
            "v"(af[ps][2]), "v"(af[ps][3]), "v"(bf[ps][0]), "v"(bf[ps][1]));
      af[slot][0] = u32x4{s0.x, s0.y, s1.x, s1.y};
      af[slot][1] = u32x4{s2.x, s2.y, s3.x, s3.y};
      af[slot][2] = u32x4{s4.x, s4.y, s5.x, s5.y};
      af[slot][3] = u32x4{s6.x, s6.y, s7.x, s7.y};
    } else if constexpr (BKM) {
      asm volatile(
          "ds_read_b64_tr_b16 %0, %4\n\t"
          "ds_read_b64_tr_b16 %1, %4 offset:2048\n\t"
          "ds_read_b64_tr_b16 %2, %5\n\t"
          "ds_read_b64_tr_b16 %3, %5 offset:2048\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(t0), "=&v"(t1), "=&v"(t2), "=&v"(t3)
          : "v"(b_addr[0] + ob), "v"(b_addr[1] + ob), "v"(af[ps][0]), "v"(af[ps][1]),
            "v"(af[ps][2]), "v"(af[ps][3]), "v"(bf[ps][0]), "v"(bf[ps][1]));
    }
    if constexpr (BKM) {
      bf[slot][0] = u32x4{t0.x, t0.y, t1.x, t1.y};
      bf[slot][1] = u32x4{t2.x, t2.y, t3.x, t3.y};
    }
  };
  TileUnit cur, nxt;
  int frags = FM;
  // DMA instruction q of the A (B) half of k-tile kt into A (B) slot `slot`.
  auto dma_one = [&](__amdgpu_buffer_rsrc_t r, int kt, int slot, bool b, int q) {
    dma16(r, &lds[((b ? 2 : 0) + slot) * SLOT + (wave * INST + q) * 64], b ? offB[q] : offA[q],
          koff(kt, b));
  };
  // The MFMAs of fragment slot s; with half >= 0 the four DMA instructions of one operand (0: A, 1: B)
  // of the unit's k-tile kt (past its last one: the next unit's) go out between the first of them.
  // PART: the row tile ends inside the block's tile, and the MFMAs of fragments of 32 rows without
  // a row to store are skipped (each SIMD holds a wave of the upper and one of the lower half).
  auto kstep = [&](int s, int kt, int slot, auto half, auto part) {
    constexpr int H = decltype(half)::value;
    constexpr bool PART = decltype(part)::value;
    const bool over = kt >= cur.KL;
    const int k = over ? kt - cur.KL : kt;
    const __amdgpu_buffer_rsrc_t r = res(over ? nxt : cur, k, H == 1);
#pragma unroll
    for (int m = 0; m < FM * FN; ++m) {
      if (!PART || m / FN < frags)
        Frag<__bf16>::mma(acc[m / FN][m % FN], bf[s][m % FN], af[s][m / FN]);
      if (H >= 0 && m < INST) dma_one(r, k, slot, H == 1, m);
    }
    if constexpr (H >= 0 && !PART) {
#pragma unroll
      for (int m = 0; m < FM * FN; ++m) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (m < INST) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
    }
  };
  using HN = std::integral_constant<int, -1>;
  using HA = std::integral_constant<int, 0>;
  using HB = std::integral_constant<int, 1>;
  // k-tile kl of the unit from A slot a, B slot b. The DMA runs ahead: the B half of k-tile kl + 2 goes
  // out in k-step 0, the A half in k-step 3, behind the barrier that frees this k-tile's slots (its
  // last fragments are in registers by then). That barrier waits for k-tile kl + 1 but not for the
  // four newest loads, the B half of kl + 2: B is the weights, read by few tiles and mostly from
  // HBM, and has 1.75 k-tiles to land; A is shared by more tiles, mostly comes from L2, and has one.
  // After a whole tile's epilogue its stores (one instruction per 16 bytes of a lane: kStores) lie
  // between those loads and k-tile kl + 1, and the first barrier leaves them in flight too.
  // (A layer's epilogue stores that much too; where it kept Z as well, or read anything, more lies between.)
  constexpr int kStores = ADD ? 0 : sizeof(TO) == 2 ? FM * FN * 2 : FM * FN * 4;
  constexpr int kVm = 4 + kStores, kLate = (kVm & 15) | (kVm >> 4) << 14 | 0x70;
  static_assert(kVm < 64, "vmcnt has six bits");
  bool late = false;
  auto body = [&](int kl, int a, int b, auto part) {
    const int b1 = b == 2 ? 0 : b + 1, b2 = b == 0 ? 2 : b - 1;
    __builtin_amdgcn_s_waitcnt(0xC07F);
    load_frags(a, b, 1, 1);
    __builtin_amdgcn_sched_barrier(0);
    kstep(0, kl + 2, b2, HB{}, part);
    __builtin_amdgcn_sched_barrier(0);
    load_tr(a, b, 1, 1);
    load_frags(a, b, 2, 0);
    __builtin_amdgcn_sched_barrier(0);
    kstep(1, 0, 0, HN{}, part);
    __builtin_amdgcn_sched_barrier(0);
    load_tr(a, b, 2, 0);
    load_frags(a, b, 3, 1);
    __builtin_amdgcn_sched_barrier(0);
    kstep(0, 0, 0, HN{}, part);
    __builtin_amdgcn_sched_barrier(0);
    load_tr(a, b, 3, 1);
    asm volatile("" ::: "memory");
    if (late) __builtin_amdgcn_s_waitcnt(kLate);
    else __builtin_amdgcn_s_waitcnt(0x0074);  // vmcnt(4) lgkmcnt(0)
    late = false;
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load_frags(a ^ 1, b1, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    kstep(1, kl + 2, a, HA{}, part);
    __builtin_amdgcn_sched_barrier(0);
    load_tr(a ^ 1, b1, 0, 0);
  };
  // The tile through LDS, so that whole 128-byte lines leave, 16 bytes a lane. The B slot of the k-tile
  // just finished (the third: the next two hold or receive the next unit's) is free until this
  // wave's own DMA fills its 4 KB of it again, so each wave stages 32 rows x 64 columns there by
  // itself, without a barrier. Chunk c of row r lies at c ^ (r >> 1 & 7), its two halves swapped in
  // rows 16 to 31: the 32 rows a half-wave writes then cover all 64 banks once.
  auto store_rows = [&](int b) {
    __bf16* out = static_cast<__bf16*>(p.C) + cur.origin;
    // Opaque here, so that the addresses below are computed now and not kept across the main loop
    // (they would be spilled, and reloading them waits for every store and DMA in flight).
    int ln = lane;
    asm volatile("" : "+v"(ln));
    __bf16* const stage = reinterpret_cast<__bf16*>(lds + (2 + b) * SLOT + wave * 256);
    const int c = ln & 7, n = wn * 64 + c * 8;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int rr = ln & 31;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int col = 32 * j + 8 * g + 4 * (ln >> 5);
          __bf16* dst = stage + rr * 64 + ((col >> 3) ^ ((rr >> 1) & 7)) * 8 +
                        ((col & 4) ^ ((rr >> 2) & 4));
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = (__bf16)acc[i][j][4 * g + e];
        }
      u32x4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = (ln >> 3) + 8 * q;
        v[q] = *reinterpret_cast<const u32x4*>(stage + r * 64 + (c ^ ((r >> 1) & 7)) * 8);
        if (q >= 2) v[q] = u32x4{v[q].z, v[q].w, v[q].x, v[q].y};
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int m = wm * 128 + 32 * i + (ln >> 3) + 8 * q;
        if (m >= cur.m_valid) continue;
        __bf16* dst = out + m * (int)p.ldc + n;
        if (n + 8 <= cur.n_valid) {
          __builtin_memcpy(dst, &v[q], 16);
        } else {
          __bf16 x[8];
          __builtin_memcpy(x, &v[q], 16);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < cur.n_valid) dst[e] = x[e];
        }
      }
    }
  };

  // A layer's epilogue: the arithmetic on the accumulators as they lie (a lane: one row, four neighbouring
  // columns of every eight), each row-wise operand and output through the same 4 KB as in store_rows, 32
  // rows x 64 columns of bfloat16 at a time. The operands of the next 32 rows are loaded before the
  // current ones are finished. Row-wise memory is reached through buffer resources that end with the
  // tile's last row, so no access is guarded by a branch: what lies outside is not read (zeros) nor
  // written, and the number of accesses in flight is known (kStores). Which operands there are and the
  // activation are compile-time (as runtime branches the accumulators spill, up to 500 bytes a lane).
  // Bound by its vector instructions, about 4 us a pass over the 16384 x 8192 elements an instruction:
  // both waves of a SIMD come to it together, so the matrix units wait. 16384 rows, 32 experts of
  // 8192 x 1024, us, one after the other in one process: forward, product 287, bias 288, + relu 294, silu 308,
  // gelu 329, + Z kept 368; with a residual relu 339, silu 360, gelu 380; input gradient, product 297,
  // none 293, relu 332 (Z's 268 MB), silu 351, gelu 381, with a residual 412.
  auto layer_rows = [&](int b) {
    if constexpr (kLayer<Args>) {
      int ln = lane;
      asm volatile("" : "+v"(ln));
      char* const stage = reinterpret_cast<char*>(lds + (2 + b) * SLOT + wave * 256);
      const int c = ln & 7, r8 = ln >> 3;
      const bool in = wn * 64 + 8 * c < cur.n_valid;       // whole chunks: p.N is a multiple of 8
      // bytes of element (row of 32, column of 64) in the stage, for 8-byte (one row a lane) and for
      // 16-byte accesses (row r8 + 8 q, whose halves are swapped from row 16 on)
      const int rr = ln & 31;
      auto own = [&](int j, int g) {
        const int k = 32 * j + 8 * g + 4 * (ln >> 5);
        return rr * 128 + ((k >> 3) ^ ((rr >> 1) & 7)) * 16 + (((k & 4) ^ ((rr >> 2) & 4)) << 1);
      };
      auto wide = [&](int q) { return (r8 + 8 * q) * 128 + (c ^ (((r8 + 8 * q) >> 1) & 7)) * 16; };
      auto rows_of = [&](const void* base, int64_t ld) {
        return make_rsrc(static_cast<const __bf16*>(base) + (int64_t)cur.row * ld + cur.col,
                         ((int64_t)(cur.m_valid < BM ? cur.m_valid - 1 : BM - 1) * ld +
                          (cur.n_valid < BN ? cur.n_valid : BN)) * 2);
      };
      // Byte offsets, below 2^30 for a tile's rows (pitches are at most 2^21); a column past the end: 7 2^28.
      // They are the lanes' as a whole, none in a scalar register: the check takes a scalar offset off the
      // resource's end first, and that of a row past a part tile's last one lies beyond it (no borrow is
      // specified).
      auto lane_at = [&](int64_t ld) { return in ? unsigned(r8 * (int)ld + 8 * c) * 2u : 0x70000000u; };
      auto row_at = [&](int64_t ld, int i, int q) {
        return unsigned((wm * 128 + 32 * i + 8 * q) * (int)ld + wn * 64) * 2u;
      };
      auto fetch = [&](const void* base, int64_t ld, int i, u32x4 (&v)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                               rows_of(base, ld), lane_at(ld) + row_at(ld, i, q), 0, 0));
      };
      auto into_stage = [&](const u32x4 (&v)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<u32x4*>(stage + wide(q)) =
              q >= 2 ? u32x4{v[q].z, v[q].w, v[q].x, v[q].y} : v[q];
      };
      auto staged = [&](int j, int g, float* x) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(stage + own(j, g));
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
      };
      auto put = [&](int i, void* base, int64_t ld) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            __bf16 t[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = (__bf16)acc[i][j][4 * g + e];
            *reinterpret_cast<u32x2*>(stage + own(j, g)) = __builtin_bit_cast(u32x2, t);
          }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u32x4 v = *reinterpret_cast<const u32x4*>(stage + wide(q));
          if (q >= 2) v = u32x4{v.z, v.w, v.x, v.y};
          // (the whole offset per lane, none in a scalar register: behind a 16-byte buffer store with one
          // the compiler lets the next instruction overwrite the store's data, and on this part that
          // instruction won)
          __builtin_amdgcn_raw_buffer_store_b128(v, rows_of(base, ld), lane_at(ld) + row_at(ld, i, q), 0, 0);
        }
      };
      // Four bias columns a lane for each of its accumulators' groups of four; with a residual's registers
      // beside them too many to keep, so loaded for every 32 rows there (from L1).
      u32x2 bias[FN][4];
      auto load_bias = [&] {
        unsigned at = 8 * (ln >> 5) + wn * 128;
        asm volatile("" : "+v"(at));       // computed here, not kept (spills of silu with a residual 112 -> 76 bytes)
        const __amdgpu_buffer_rsrc_t r =
            make_rsrc(static_cast<const __bf16*>(p.bias) + (int64_t)cur.expert * p.N + cur.col,
                      p.bias ? (cur.n_valid < BN ? cur.n_valid : BN) * 2 : 0);
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            bias[j][g] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                                                       r, at + (32 * j + 8 * g) * 2, 0, 0));
      };
      constexpr bool gate = FORM == NN && ACT != ACT_NONE;
      u32x4 ahead[4];
      if (gate) fetch(p.Z, p.ldz, 0, ahead);
      else if (RES) fetch(p.R, p.ldr, 0, ahead);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if constexpr (FORM == NT) {
          if (RES || i == 0) load_bias();
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              acc[i][j][4 * g] += __uint_as_float(bias[j][g].x << 16);
              acc[i][j][4 * g + 1] += __uint_as_float(bias[j][g].x & 0xFFFF0000u);
              acc[i][j][4 * g + 2] += __uint_as_float(bias[j][g].y << 16);
              acc[i][j][4 * g + 3] += __uint_as_float(bias[j][g].y & 0xFFFF0000u);
            }
          if constexpr (KEEP) put(i, p.Z, p.ldz);
        } else if constexpr (gate) {
          into_stage(ahead);
          if (RES) fetch(p.R, p.ldr, i, ahead);
          else if (i + 1 < FM) fetch(p.Z, p.ldz, i + 1, ahead);
        }
#pragma unroll
        for (int h = 0; h < 2 * FN; ++h) {
          float v[8], x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = acc[i][h / 2][8 * (h % 2) + e];
          if constexpr (FORM == NT) {
            activate<false>(ACT, v);
          } else if constexpr (gate) {
            staged(h / 2, 2 * (h % 2), x);
            staged(h / 2, 2 * (h % 2) + 1, x + 4);
            times_slope<false>(ACT, v, x);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[i][h / 2][8 * (h % 2) + e] = v[e];
        }
        if constexpr (RES) {
          into_stage(ahead);
          if (i + 1 < FM) {
            if (gate) fetch(p.Z, p.ldz, i + 1, ahead);
            else fetch(p.R, p.ldr, i + 1, ahead);
          }
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float t[4];
              staged(j, g, t);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][4 * g + e] += t[e];
            }
        }
        put(i, p.C, p.ldc);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // The same with beta C, added to the float32 sum (one rounding): a fragment of 32 x 32 at a time,
  // whose addend is loaded while it goes through LDS. (A float32 output without an addend is
  // stored from registers, two lanes a 32-byte piece: 470 against 479 us on 32 experts of
  // 8192 x 1024; with one, pieces took 640 us and whole lines take 593.)
  auto store_sums = [&](int b) {
    TO* out = static_cast<TO*>(p.C) + cur.origin;
    const TO* D = static_cast<const TO*>(p.D) + cur.origin;
    int ln = lane;
    asm volatile("" : "+v"(ln));
    floatx4* const stage = reinterpret_cast<floatx4*>(lds + (2 + b) * SLOT + wave * 256);
    const int c = ln & 7, r0 = ln >> 3;
#pragma unroll
    for (int f = 0; f < FM * FN; ++f) {
      const int n = wn * 64 + 32 * (f % FN) + 4 * c, m0 = wm * 128 + 32 * (f / FN) + r0;
      TO add[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // past the last row: the tile's first, in bounds and not used
        const TO* src = D + (m0 + 8 * q < cur.m_valid ? (m0 + 8 * q) * (int)p.ldc : 0) + n;
        if (n + 4 <= cur.n_valid) {
          __builtin_memcpy(add[q], src, sizeof(add[q]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) add[q][e] = n + e < cur.n_valid ? src[e] : (TO)0.f;
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        floatx4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[f / FN][f % FN][4 * g + e];
        stage[(ln & 31) * 8 + ((2 * g + (ln >> 5)) ^ ((ln >> 1) & 7))] = v;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = r0 + 8 * q;
        const floatx4 v = stage[r * 8 + (c ^ ((r >> 1) & 7))];
        if (m0 + 8 * q >= cur.m_valid) continue;
        TO t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = (TO)(v[e] + p.beta * (float)add[q][e]);
        TO* dst = out + (m0 + 8 * q) * (int)p.ldc + n;
        if (n + 4 <= cur.n_valid) {
          __builtin_memcpy(dst, t, sizeof(t));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < cur.n_valid) dst[e] = t[e];
        }
      }
    }
  };

  clear();
  if (unit(0, cur)) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {               // B 0, A 0, B 1, A 1
      const __amdgpu_buffer_rsrc_t r = res(cur, h >> 1, !(h & 1));
#pragma unroll
      for (int q = 0; q < INST; ++q) dma_one(r, h >> 1, h >> 1, !(h & 1), q);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) af[1][i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[1][j] = u32x4{0u, 0u, 0u, 0u};
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0078);         // vmcnt(8): k-tile 0 has landed
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load_frags(0, 0, 0, 0);
    load_tr(0, 0, 0, 0);
    int a = 0, b = 0;
    bool more = true;
    for (int i = 1; more; ++i) {
      more = unit(i, nxt);
      if (!more) {                // nothing follows: the DMA past the end reads no bytes
        nxt = cur;
        nxt.a_bytes = nxt.b_bytes = 0;
        nxt.rows = 0;
      }
      const int below = cur.m_valid - 128 * wm;
      frags = below <= 0 ? 0 : below >= 128 ? FM : (below + 31) / 32;
      auto run = [&](auto part) {
        for (int kl = 0; kl < cur.KL; ++kl) {
          body(kl, a, b, part);
          a ^= 1;
          b = b == 2 ? 0 : b + 1;
        }
      };
      if (cur.m_valid >= BM) run(std::false_type{});
      else run(std::true_type{});
      if (cur.slot >= 0) {
        floatx4* P = reinterpret_cast<floatx4*>(p.partial) + (int64_t)cur.slot * (BM * BN / 4);
#pragma unroll
        for (int m = 0; m < FM * FN; ++m)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            floatx4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[m / FN][m % FN][4 * g + e];
            P[(m * 4 + g) * 512 + tid] = v;
          }
      } else if constexpr (kLayer<Args>) {
        layer_rows(b == 0 ? 2 : b - 1);
      } else if constexpr (ADD) {
        store_sums(b == 0 ? 2 : b - 1);
      } else if constexpr (sizeof(TO) == 2) {
        store_rows(b == 0 ? 2 : b - 1);
      } else {
        store_fragments<TO, FM, FN, false>(p, acc, cur.origin, wm * 128, wn * 64, cur.m_valid,
                                           cur.n_valid);
      }
      late = !ADD && cur.slot < 0 && (kLayer<Args> || (cur.m_valid >= BM && cur.n_valid >= BN));
      clear();
      // the next tile's first fragments again: they need not stay in registers over the epilogue
      if constexpr (kLayer<Args> && FORM == NT) load_frags(a, b, 0, 0);
      cur = nxt;
    }
    block_sync();                 // no DMA is in flight when the block ends
  }
  // The rows of no expert: before the first one's begin and from the last one's end.
  if (FORM != TN && p.fill_rest) {
    int first, last, x;
    expert_rows(p, 0, first, x);
    expert_rows(p, p.groups - 1, x, last);
    const int rest = first + (p.total_rows - last);
    __bf16* out = static_cast<__bf16*>(p.C);
    for (int r = blockIdx.x; r < rest; r += gridDim.x) {
      const int64_t row = r < first ? r : last + (r - first);
      for (int n = tid * 8; n < p.N; n += 512 * 8) {
        if (n + 8 <= p.N) {
          const u32x4 z = {0u, 0u, 0u, 0u};
          __builtin_memcpy(out + row * p.ldc + n, &z, 16);
          if constexpr (kLayer<Args> && FORM == NT) {      // (p.N is a multiple of 8 there)
            if (KEEP) __builtin_memcpy(static_cast<__bf16*>(p.Z) + row * p.ldz + n, &z, 16);
          }
        } else {
          for (int e = n; e < p.N; ++e) out[row * p.ldc + e] = (__bf16)0.f;
        }
      }
    }
  }
}

// Adds the parts of the last round's split tiles in part order and stores them: one block per
// 64 x 64 piece of a tile (the product kernel's fragment order: float4 (m * 4 + g) * 512 + thread).
// Bound by reading the parts from memory: 3 to 15 us, 64 MB of them at most.
template <typename TO, int FORM, typename Args>
__global__ __launch_bounds__(256) void k_grouped_join(Args p) {
  Walk walk = {};
  int rank = -1;
  if constexpr (FORM == TN) {
    if (p.groups <= 64) rank = rows_rank(p);
    walk.total = (p.N + 255) / 256 * p.tiles_n * p.groups;
  } else {
    walk = walk_start(p, 256, p.tiles_n, 0);
  }
  const Deal dl = deal(walk.total, p.split_cap);
  const int t = blockIdx.x >> 4, piece = blockIdx.x & 15;
  if (dl.split < 2 || t >= dl.tail) return;
  int expert, lo, hi, m0, n0;
  if (!tile_at<FORM>(p, walk, rank, dl.rounds * 256 + t, expert, lo, hi, m0, n0)) return;
  const int m_valid = FORM == TN ? p.N - m0 : hi - m0;
  const int n_valid = (FORM == TN ? p.K : p.N) - n0;
  // this piece's fragments: rows 64 (piece / 4) .., columns 64 (piece % 4) ..
  const int wm = piece >> 3, wn = piece & 3, i0 = ((piece >> 2) & 1) * 2;
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;       // wave q: fragment (i0 + q / 2, q % 2)
  const floatx4* P = reinterpret_cast<const floatx4*>(p.partial) +
                     (((i0 + q / 2) * 2 + q % 2) * 4) * 512 + (wm * 4 + wn) * 64 + lane;
  const int pm = wm * 128 + 32 * (i0 + q / 2), pn = wn * 64 + 32 * (q % 2);
  FinishOf<Args, TO, FORM, 1, 1> end(expert, m0, n0, pm, pn, m_valid, n_valid);
  if constexpr (kLayer<Args>) end.load_first(p);
  floatx16 acc[1][1];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[0][0][e] = 0.f;
  for (int part = 0; part < dl.split; ++part) {
    const floatx4* src = P + (int64_t)(part * dl.tail + t) * (256 * 256 / 4);
    floatx4 v[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) v[g] = src[g * 512];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][0][4 * g + e] += v[g][e];
  }
  if constexpr (kLayer<Args>) {
    __shared__ floatx4 stage[4 * 256];
    end.run(p, acc, stage + q * 256);
  } else {
    store_fragments<TO, 1, 1, FORM == TN>(p, acc, (FORM == TN ? expert * p.sC : 0) + m0 * p.ldc + n0,
                                          pm, pn, m_valid, n_valid);
  }
}

// ---- a middling number of rows, bfloat16 ------------------------------------------------------
//
// Also for more rows whose 256 x 256 tiles would leave most CUs without work (plan_of).
// Up to some hundred rows per expert the weights' bytes still bound a forward or input gradient,
// and the rows fit one or two tiles of 128: a block takes 128 rows x BN columns, so most weights
// are read once. What counts is bytes in flight: a ring of NS k-tiles in LDS (160 KB a CU), all but
// one of them loading, one barrier per k-tile. 512 rows over 8 experts of 4096 x 2048: 34 us, 4.1 TB/s,
// in one round of 256 blocks, whose first and last k-tiles nothing overlaps. Fragments of 32 rows
// without a row are skipped;
// operand layouts as in k_grouped_big (a [k][BN] operand with BN = 64 has chunk c of k-row r at
// c ^ 4 (r >> 1 & 1)).
template <int FORM, int BN, typename Args>
__global__ __launch_bounds__(256) void k_grouped_ring(Args p) {
  constexpr int BM = 128, BK = 64, FM = 2, FN = BN / 64, AI = 4, BI = BN / 32;
  constexpr bool BKM = FORM == NN;
  constexpr int NS = BN == 128 ? 5 : 6;
  constexpr int STAGE = (BM + BN) * kChunks;
  constexpr int KCH = BN / 8, KROW = BN * 2;            // chunks and bytes of a [k][BN] row
  __shared__ u32x4 lds[NS * STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  Place at;
  if (!find_place(p, BM, p.tiles_n, p.fill_rest, walk_start(p, BM, p.tiles_n, p.fill_rest),
                  block_place(), at))
    return;
  const int m0 = at.lo + at.inside / p.tiles_n * BM, n0 = at.inside % p.tiles_n * BN;
  const int m_valid = at.hi - m0, n_valid = p.N - n0;
  if constexpr (kLayer<Args>) {
    if (at.expert < 0) {
      zero_tile<__bf16, FORM>(p, m0, n0, m_valid < BM ? m_valid : BM, n_valid < BN ? n_valid : BN);
      return;
    }
  }
  const int KL = at.expert < 0 ? 0 : p.K / BK;
  FinishOf<Args, __bf16, FORM, FM, FN> end(at.expert, m0, n0, wm * 64, wn * (BN / 2), m_valid, n_valid);
  if constexpr (kLayer<Args>) end.load_first(p);

  floatx16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  if (KL > 0) {
    const __amdgpu_buffer_rsrc_t rA =
        make_rsrc(static_cast<const char*>(p.A) + m0 * p.lda * 2,
                  ((int64_t)((m_valid < BM ? m_valid : BM) - 1) * p.lda + p.K) * 2);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(
        static_cast<const char*>(p.B) + (at.expert * p.sB + (BKM ? (int64_t)n0 : n0 * p.ldb)) * 2,
        (BKM ? (int64_t)p.K * p.ldb - n0 : (int64_t)n_valid * p.ldb) * 2);
    const __amdgpu_buffer_rsrc_t none = make_rsrc(p.A, 0);     // reads zeros from nowhere
    int offA[AI], offB[BI];
#pragma unroll
    for (int i = 0; i < AI; ++i) {
      const int row = (wave * AI + i) * 8 + (lane >> 3);
      offA[i] = (row * (int)p.lda + 8 * ((lane & 7) ^ ((row ^ ((row >> 3) & 3)) & 7))) * 2;
    }
#pragma unroll
    for (int i = 0; i < BI; ++i) {
      if constexpr (BKM) {
        const int kr = (64 / KCH) * (wave * BI + i) + lane / KCH;
        const int x = BN == 128 ? 4 * (kr & 3) : 4 * ((kr >> 1) & 1);
        offB[i] = (kr * (int)p.ldb + 8 * ((lane % KCH) ^ x)) * 2;
      } else {
        const int row = (wave * BI + i) * 8 + (lane >> 3);
        offB[i] = (row * (int)p.ldb + 8 * ((lane & 7) ^ ((row ^ ((row >> 3) & 3)) & 7))) * 2;
      }
    }
    auto issue = [&](int kt, int st) {
      const bool real = kt < KL;
      const __amdgpu_buffer_rsrc_t a = real ? rA : none, b = real ? rB : none;
      const int ka = real ? kt * BK * 2 : 0, kb = !real ? 0 : BKM ? kt * BK * (int)p.ldb * 2 : ka;
#pragma unroll
      for (int i = 0; i < BI; ++i)
        dma16(b, &lds[st * STAGE + BM * kChunks + (wave * BI + i) * 64], offB[i], kb);
#pragma unroll
      for (int i = 0; i < AI; ++i)
        dma16(a, &lds[st * STAGE + (wave * AI + i) * 64], offA[i], ka);
    };
    const int below = m_valid - 64 * wm;
    const int frags = below <= 0 ? 0 : below > 32 ? 2 : 1;
    uint32_t b_addr[FN] = {};
    if constexpr (BKM) {
      const int G = lane >> 4, sq = (lane & 15) >> 2, a4 = lane & 3, kb = 8 * (G >> 1) + sq;
      const int x = BN == 128 ? 4 * (kb & 3) : 4 * ((kb >> 1) & 1);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int c = wn * (BN / 2) + 32 * j + 16 * (G & 1) + 4 * a4;
        b_addr[j] = lds_address(lds) + BM * 128 + kb * KROW + ((c >> 3) ^ x) * 16 + (c & 7) * 2;
      }
    }
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) issue(s, s);
    int st = 0, fill = NS - 1;
    for (int kt = 0; kt < KL; ++kt) {
      // k-tile kt has landed (NS - 2 newer ones may be on their way), for every wave behind the
      // barrier, where the stage of k-tile kt - 1 is free too
      constexpr int kVm = (NS - 2) * (AI + BI);
      static_assert(kVm < 64, "vmcnt has six bits");
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt((kVm & 15) | (kVm >> 4) << 14 | 0x70);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      issue(kt + NS - 1, fill);
      const u32x4* A = lds + st * STAGE;
      const u32x4* B = A + BM * kChunks;
      u32x4 a[4][FM], b[4][FN];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int ch = 2 * ks + (lane >> 5);
#pragma unroll
        for (int i = 0; i < FM; ++i) a[ks][i] = A[swz(wm * 64 + 32 * i + (lane & 31), ch)];
        if constexpr (!BKM) {
#pragma unroll
          for (int j = 0; j < FN; ++j)
            b[ks][j] = B[swz(wn * (BN / 2) + 32 * j + (lane & 31), ch)];
        }
      }
      if constexpr (BKM) {
        // one k-tile's transposing reads of a fragment column, waited for in the same block (the
        // compiler would wait for every outstanding DMA)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const uint32_t at0 = b_addr[j] + (uint32_t)(st * STAGE * 16);
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
              : "v"(at0), "i"(4 * KROW), "i"(16 * KROW), "i"(20 * KROW), "i"(32 * KROW),
                "i"(36 * KROW), "i"(48 * KROW), "i"(52 * KROW));
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            b[ks][j] = u32x4{t[2 * ks].x, t[2 * ks].y, t[2 * ks + 1].x, t[2 * ks + 1].y};
        }
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
        if (i < frags) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int j = 0; j < FN; ++j) Frag<__bf16>::mma(acc[i][j], b[ks][j], a[ks][i]);
        }
      st = st + 1 == NS ? 0 : st + 1;
      fill = fill + 1 == NS ? 0 : fill + 1;
    }
    block_sync();                 // no DMA is in flight when the block ends
  }
  if constexpr (kLayer<Args>)
    end.run(p, acc, reinterpret_cast<floatx4*>(lds) + wave * 256);
  else
    store_fragments<__bf16, FM, FN, false>(p, acc, m0 * p.ldc + n0, wm * 64, wn * (BN / 2), m_valid,
                                           n_valid);
}

// Whether rows of a bfloat16 W start between two dwords (early).
bool between_dwords(const GroupedArgs& a) {
  return (reinterpret_cast<uintptr_t>(a.B) & 2) || (a.ldb & 1);
}

template <typename T, typename TO, int FORM, typename Args>
hipError_t launch_grouped(const Args& a, int64_t blocks, hipStream_t s) {
  const dim3 grid = grid_of(blocks), block(256);
  if constexpr (FORM == NN && sizeof(T) == 2) {
    if (between_dwords(a)) {
      hipLaunchKernelGGL((k_grouped<T, TO, FORM, Args, true>), grid, block, 0, s, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_grouped<T, TO, FORM, Args, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <typename T, typename Args>
hipError_t launch_split(const Args& a, bool transpose_w, int64_t blocks, hipStream_t s) {
  const dim3 block(256);
  dim3 grid = grid_of(blocks);
  if constexpr (kLayer<Args>) grid = grid_of(blocks * a.parts);
  if (!transpose_w) hipLaunchKernelGGL((k_grouped_split<T, NT, Args, false>), grid, block, 0, s, a);
  else if (sizeof(T) == 2 && between_dwords(a))
    hipLaunchKernelGGL((k_grouped_split<T, NN, Args, sizeof(T) == 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_grouped_split<T, NN, Args, false>), grid, block, 0, s, a);
  const hipError_t e = hipGetLastError();
  if constexpr (kLayer<Args>) {
    if (e != hipSuccess || a.parts == 1) return e;
    grid = grid_of(blocks);
    if (transpose_w) hipLaunchKernelGGL((k_split_join<T, NN>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_split_join<T, NT>), grid, block, 0, s, a);
    return hipGetLastError();
  }
  return e;
}

int64_t tiles_up(int64_t x, int64_t t) { return (x + t - 1) / t; }

int cu_count() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) == hipSuccess &&
        hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && v > 0)
      return v;
    return 256;
  }();
  return n;
}

// Most 64 x 64 tiles of rows that belong to an expert.
int64_t split_tiles(const GroupedDesc& d) {
  return (std::min(d.groups, d.total_rows) + d.total_rows / 64) *
         tiles_up(d.transpose_w ? d.k : d.n, 64);
}

// Tile and kernel of a call, from its sizes alone.
enum class Kernel { Tile128, Split64, Rows, Ring, Big };
struct Plan {
  Kernel kernel;
  int bm, bn;           // output tile
  int mt, ntw, wk;      // Rows
};

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// What the DMA kernels assume: bfloat16, 16-byte aligned operands and row pitches, a whole number of
// k-tiles (the weight gradient's reduction may end anywhere), and for W read along the output one
// expert's matrix below 2 GiB. The weight gradient's resources end with the last row's last element,
// and the hardware checks a load dword by dword: one that an odd width ends inside of would read as
// zero, last element and all, so its widths are even.
bool dma_ok(const GroupedDesc& d) {
  if (d.store != Store::BF16 || !on16(d.A) || !on16(d.B) || d.lda % 8) return false;
  if (d.weight_grad) return d.ldb % 8 == 0 && d.n % 2 == 0 && d.k % 2 == 0;
  const int64_t red = d.transpose_w ? d.n : d.k;
  // a layer's epilogue moves whole chunks, and four bias elements a load, which must start on a dword
  if (d.layer && ((d.transpose_w ? d.k : d.n) % 8 || !on16(d.C) || !on16(d.R) || !on16(d.Z) ||
                  (reinterpret_cast<uintptr_t>(d.bias) & 3) ||
                  d.ldc % 8 || (d.R && d.ldr % 8) || (d.Z && d.ldz % 8)))
    return false;
  return red % 64 == 0 && red >= 128 && d.k % 8 == 0 && (d.n * d.k) % 8 == 0 &&
         d.n * d.k < (int64_t(1) << 30);
}

// The kernel of a call, by sizes, types and alignment. Times in us of random rows per expert
// ("4096x2048 x 8": 8 experts of n = 4096, k = 2048; weights not in a cache):
//
//   Weight gradient without an addend: k_grouped_big whenever its DMA applies (against k_grouped, 24
//   rows each: 121 / 212 on 8192x1024 x 32, 41 / 52 on 4096x2048 x 8, 20 / 20 on 1024x4096 x 4).
//   With one the addend and the output are what is moved, and many small tiles keep more of it in
//   flight: k_grouped up to 128 rows each (24 rows: 401 / 473 of k_grouped_big, 107 / 126,
//   34 / 38; 128 rows: 461 / 490, 127 / 127, 39 / 37; 512 rows: 919 / 615, 225 / 164, 62 / 47).
//   Forward, input gradient: k_grouped_big from 448 tiles of 256 x 256 on, whatever the rows: its
//   blocks run from tile to tile without a break, so the weights stream at the HBM rate (8192x1024
//   x 32, forward: 12 rows 103 against 118 of k_grouped_ring and 133 of k_grouped_rows, 100 rows
//   125 / 160 / 248; input gradient, 128 tiles, so not by this rule: 12 rows 122 / 97).
//   Fewer tiles leave CUs without work for too long; then, forward with at most 24 rows each,
//   k_grouped_rows (4096x2048 x 8, 12 rows: 35 against 38 of k_grouped_ring and 48 of
//   k_grouped_big; 1024x4096 x 4: 16 / 30 / 26; 40 rows: 41 / 40 / 51 and 20 / 35 / 27), else
//   k_grouped_ring up to 256 rows each (4096x2048 x 8, 100 rows: 41 / 52 of k_grouped_big; input
//   gradient 12 rows 43 / 52, 100 rows 57 / 55) if it has a block for every other CU or the
//   reduction is too short for k_grouped_big to split; beyond, k_grouped_big (300 rows: 54 / 92 of
//   k_grouped_ring, input gradient 74 / 113) unless its grid is small: where tiles of k_grouped_ring
//   fill about one round and the reduction is at most 2048, those (in a cache; one expert of 2048 rows,
//   512x1024: 14 of k_grouped_ring / 24, 1024x2048 30 / 32, 512x4096 37 / 30; four of 1024, 512x512
//   13 / 16, of 300, 2048x512 13 / 16, of 2048, 1024x512, two rounds, 28 / 18; over 734 sizes of 1 to 8
//   experts of 300 to 8192 rows 2 % from the faster of the two, k_grouped_big alone 23 %).
//   A layer of few tiles of 64 x 64 and a long reduction: k_grouped_split in parts (split_parts), with
//   operands for the DMA too. Its time over that of k_grouped_ring or k_grouped_big, split or not (252 sizes
//   of 1 to 16 experts, means for up to 64 / 128 / 256 tiles): input gradients, reduction 1024 1.15 / 1.24 /
//   1.38, 2048 0.79 / 0.87 / 1.08, 4032 0.82 / 0.90 / 1.06, 8192 0.85 / 1.01 / 1.11; forwards 0.84 / 1.02 / 1.19 (26
//   rows an expert: 1.2), 0.68 / 0.85 / 1.02, 0.81 / 0.99 / 1.05, 0.95 / 1.20 / 1.19 (us: 7 experts, 1 row, input
//   gradient of 4992 x 1152 16.6 / 24.2; 58, 909 rows, 2560 x 64 16.8 / 32.8; 3, 624 rows, forward of 192 x 3968
//   20.1 / 24.2).
//   What the DMA cannot take: k_grouped_rows up to 96 rows each (forward); k_grouped_split up to 160
//   tiles of 128 x 128 (float32, 1021 rows over 5 experts of 513x1277: forward 36 against 103,
//   input gradient 37 / 47; bfloat16 45 / 62 and 26 / 26; 200 tiles: 142 / 124, 51 / 38), else
//   k_grouped.
Plan plan_of(const GroupedDesc& d) {
  Plan p{Kernel::Tile128, 128, 128, 0, 0, 0};
  const bool dma = dma_ok(d);
  const int64_t cus = cu_count();
  const int64_t used = d.groups < d.total_rows ? d.groups : d.total_rows;   // experts with rows
  if (d.weight_grad) {
    if (dma && (!d.D || d.total_rows > 128 * d.groups)) {
      p.kernel = Kernel::Big;
      p.bm = p.bn = 256;
    }
    return p;
  }
  const int64_t out = d.transpose_w ? d.k : d.n, red = d.transpose_w ? d.n : d.k;
  if (dma) {
    const int64_t big_tiles = (used + d.total_rows / 256) * tiles_up(out, 256);
    const int64_t bn = tiles_up(out, 128) * used >= cus / 2 ? 128 : 64;
    const int64_t ring_tiles = (used + d.total_rows / 128) * tiles_up(out, bn);
    const bool few = !d.transpose_w && d.total_rows <= 24 * used;
    const bool many = d.total_rows > 256 * d.groups;
    const bool middling = red <= 4096;
    if (d.layer && !few && (d.transpose_w && middling ? 2 : 4) * split_tiles(d) <= cus &&
        (d.transpose_w ? red >= 2048 : red >= 1536 && middling)) {
      p.kernel = Kernel::Split64;
      p.bm = p.bn = 64;
      return p;
    }
    if (many && red <= 2048) {
      const int64_t row_tiles = used + d.total_rows / 128;
      p.bn = out <= 64 || row_tiles * tiles_up(out, 64) <= cus ? 64 : 128;
      if (8 * row_tiles * tiles_up(out, p.bn) <= 9 * cus) {
        p.kernel = Kernel::Ring;
        return p;
      }
    }
    if (4 * big_tiles >= 7 * cus || many || (!few && 2 * ring_tiles < cus && red >= 1536)) {
      p.kernel = Kernel::Big;
      p.bm = p.bn = 256;
      return p;
    }
    if (!few) {
      p.kernel = Kernel::Ring;
      p.bn = (int)bn;
      return p;
    }
  }
  if (!d.transpose_w && d.total_rows <= 96 * d.groups) {
    p.kernel = Kernel::Rows;
    const int64_t avg = tiles_up(d.total_rows, used > 0 ? used : 1);
    p.mt = avg <= 16 ? 1 : avg <= 32 ? 2 : 4;
    // Eight waves per CU: 256 weight rows per block, else 64, else 16 with the reduction split.
    const int64_t row_tiles = used + d.total_rows / (16 * p.mt) / 2;
    const int64_t want = 2 * cus;                            // blocks of four waves
    if (row_tiles * tiles_up(d.n, 256) >= want) p.ntw = 4, p.wk = 1;
    else if (row_tiles * tiles_up(d.n, 64) >= want) p.ntw = 4, p.wk = 4;
    else p.ntw = 1, p.wk = 4;
    p.bm = 16 * p.mt;
    p.bn = 16 * p.ntw * (4 / p.wk);
  } else if ((used + d.total_rows / 128) * tiles_up(out, 128) <= 5 * cus / 8) {
    p.kernel = Kernel::Split64;
    p.bm = p.bn = 64;
  }
  return p;
}

template <typename T, int MT, typename Args>
hipError_t launch_rows(const Args& a, const Plan& p, int64_t blocks, hipStream_t s) {
  const dim3 grid = grid_of(blocks), block(256);
  if (p.ntw == 4 && p.wk == 1)
    hipLaunchKernelGGL((k_grouped_rows<T, MT, 4, 1, Args>), grid, block, 0, s, a);
  else if (p.ntw == 4)
    hipLaunchKernelGGL((k_grouped_rows<T, MT, 4, 4, Args>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_grouped_rows<T, MT, 1, 4, Args>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <typename T, typename Args>
hipError_t launch_rows(const Args& a, const Plan& p, int64_t blocks, hipStream_t s) {
  if (p.mt == 1) return launch_rows<T, 1>(a, p, blocks, s);
  if (p.mt == 2) return launch_rows<T, 2>(a, p, blocks, s);
  return launch_rows<T, 4>(a, p, blocks, s);
}

}  // namespace

int64_t grouped_blocks(const GroupedDesc& d) {
  const Plan p = plan_of(d);
  if (d.weight_grad) return d.groups * tiles_up(d.n, p.bm) * tiles_up(d.k, p.bn);
  // every expert with rows can end in a part tile, and so can the rows of no expert
  const int64_t ends = p.kernel == Kernel::Big ? d.groups : std::min(d.groups, d.total_rows);
  return (tiles_up(d.total_rows, p.bm) + ends + 2) * tiles_up(d.transpose_w ? d.k : d.n, p.bn);
}

// Parts of a layer's reduction on k_grouped_split: as many as fill the CUs' two blocks each, of at least 5
// k-tiles, where there are 16 or more (input gradients, us, in parts / not: float32, 141 rows over 2 experts of
// 6080 x 320 30.6 / 167, 65 of 640 x 320, 20 k-tiles, 14.9 / 23.5; bfloat16, 2 experts, 300 rows, 2500 x 1001
// 22.2 / 37; parts of at least 4 and 8 k-tiles: 46 k-tiles 16.0 and 16.8, 56 20.1 and 18.3).
static int split_parts(const GroupedDesc& d) {
  if (!d.layer || plan_of(d).kernel != Kernel::Split64) return 1;
  const int64_t k_tiles = tiles_up(d.transpose_w ? d.n : d.k, d.store == Store::F32 ? 32 : 64);
  if (k_tiles < 16) return 1;
  const int64_t parts = std::min(2 * (int64_t)cu_count() / split_tiles(d), std::min<int64_t>(k_tiles / 5, 16));
  return parts < 2 ? 1 : (int)parts;
}

template <typename TO, int FORM, int ACT>
static void launch_layer(const LayerArgs& a, hipStream_t s) {
  const dim3 grid(256), block(512);
  if constexpr (FORM == NT && ACT != ACT_NONE) {
    if (a.Z && a.R) {
      hipLaunchKernelGGL((k_grouped_big<TO, FORM, false, LayerArgs, ACT, true, true>), grid, block, 0, s, a);
      return;
    }
    if (a.Z) {
      hipLaunchKernelGGL((k_grouped_big<TO, FORM, false, LayerArgs, ACT, true, false>), grid, block, 0, s, a);
      return;
    }
  }
  if (a.R)
    hipLaunchKernelGGL((k_grouped_big<TO, FORM, false, LayerArgs, ACT, false, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_grouped_big<TO, FORM, false, LayerArgs, ACT, false, false>), grid, block, 0, s, a);
}

template <typename TO, int FORM, typename Args>
static hipError_t launch_big(const Args& a, hipStream_t s) {
  const dim3 grid(256), block(512);
  if constexpr (kLayer<Args>) {
    if (a.act == ACT_RELU) launch_layer<TO, FORM, ACT_RELU>(a, s);
    else if (a.act == ACT_RELU2) launch_layer<TO, FORM, ACT_RELU2>(a, s);
    else if (a.act == ACT_GELU) launch_layer<TO, FORM, ACT_GELU>(a, s);
    else if (a.act == ACT_SILU) launch_layer<TO, FORM, ACT_SILU>(a, s);
    else launch_layer<TO, FORM, ACT_NONE>(a, s);
  } else if (FORM == TN && a.D) {
    hipLaunchKernelGGL((k_grouped_big<TO, FORM, FORM == TN, Args>), grid, block, 0, s, a);
  } else {
    hipLaunchKernelGGL((k_grouped_big<TO, FORM, false, Args>), grid, block, 0, s, a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.split_cap < 2) return e;
  // a split last round has at most 128 tiles
  hipLaunchKernelGGL((k_grouped_join<TO, FORM, Args>), dim3(128 * 16), dim3(256), 0, s, a);
  return hipGetLastError();
}

// Parts a tile of the last round may be cut into: at least 8 k-tiles each (on the average expert,
// for the weight gradient), and only where a call has few rounds and three parts are possible, so
// that filling the last one pays for the second launch (4 to 14 us).
static int split_cap(const GroupedDesc& d) {
  const Plan p = plan_of(d);
  if (p.kernel != Kernel::Big || grouped_blocks(d) > 6 * 256) return 1;
  const int64_t red = d.weight_grad ? d.total_rows / d.groups : d.transpose_w ? d.n : d.k;
  const int64_t cap = red / 64 / 8;
  return cap < 3 ? 1 : cap > 16 ? 16 : (int)cap;
}

size_t grouped_workspace(const GroupedDesc& d) {
  if (split_cap(d) > 1) return size_t(256) * 256 * 256 * sizeof(float);
  const int parts = split_parts(d);
  return parts > 1 ? (size_t)split_tiles(d) * parts * 64 * 64 * sizeof(float) : 0;
}

const char* grouped_name(const GroupedDesc& d) {
  const bool f = d.store == Store::F32;
  switch (plan_of(d).kernel) {
    case Kernel::Rows: return f ? "grouped_rows_f32" : "grouped_rows_bf16";
    case Kernel::Ring: return d.transpose_w ? "grouped_ring_nn" : "grouped_ring_nt";
    case Kernel::Big:
      return d.weight_grad ? "grouped_256_tn" : d.transpose_w ? "grouped_256_nn" : "grouped_256_nt";
    case Kernel::Split64:
      if (d.transpose_w) return f ? "grouped_64_nn_f32" : "grouped_64_nn_bf16";
      return f ? "grouped_64_nt_f32" : "grouped_64_nt_bf16";
    default:
      if (d.weight_grad) return f ? "grouped_128_tn_f32" : "grouped_128_tn_bf16";
      if (d.transpose_w) return f ? "grouped_128_nn_f32" : "grouped_128_nn_bf16";
      return f ? "grouped_128_nt_f32" : "grouped_128_nt_bf16";
  }
}

// A forward or input gradient: the plan's kernel, with or without a layer's epilogue.
template <typename Args>
static hipError_t launch_rowwise(const GroupedDesc& d, const Plan& pl, const Args& a, int64_t blocks,
                                 hipStream_t s) {
  if (pl.kernel == Kernel::Rows)
    return d.store == Store::F32 ? launch_rows<float>(a, pl, blocks, s)
                                 : launch_rows<__bf16>(a, pl, blocks, s);
  if (pl.kernel == Kernel::Split64)
    return d.store == Store::F32 ? launch_split<float>(a, d.transpose_w, blocks, s)
                                 : launch_split<__bf16>(a, d.transpose_w, blocks, s);
  if (pl.kernel == Kernel::Ring) {
    const dim3 grid = grid_of(blocks), block(256);
    if (d.transpose_w && pl.bn == 128)
      hipLaunchKernelGGL((k_grouped_ring<NN, 128, Args>), grid, block, 0, s, a);
    else if (d.transpose_w)
      hipLaunchKernelGGL((k_grouped_ring<NN, 64, Args>), grid, block, 0, s, a);
    else if (pl.bn == 128)
      hipLaunchKernelGGL((k_grouped_ring<NT, 128, Args>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((k_grouped_ring<NT, 64, Args>), grid, block, 0, s, a);
    return hipGetLastError();
  }
  if (pl.kernel == Kernel::Big)
    return d.transpose_w ? launch_big<__bf16, NN>(a, s) : launch_big<__bf16, NT>(a, s);
  if (d.store == Store::F32)
    return d.transpose_w ? launch_grouped<float, float, NN>(a, blocks, s)
                         : launch_grouped<float, float, NT>(a, blocks, s);
  return d.transpose_w ? launch_grouped<__bf16, __bf16, NN>(a, blocks, s)
                       : launch_grouped<__bf16, __bf16, NT>(a, blocks, s);
}

hipError_t grouped(const GroupedDesc& d, hipStream_t s) {
  const Plan pl = plan_of(d);
  const int64_t blocks = grouped_blocks(d);
  if (blocks < 1 || blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  LayerArgs layer;
  GroupedArgs& a = layer;
  a.A = d.A; a.B = d.B; a.D = d.D; a.C = d.C;
  a.lda = d.lda;
  a.offsets = d.offsets;
  a.total_rows = (int)d.total_rows;
  a.groups = (int)d.groups;
  a.most_tiles = (int)blocks;
  a.fill_rest = d.fill_rest ? 1 : 0;
  a.beta = d.beta;
  a.sB = a.sC = d.n * d.k;
  a.split_cap = split_cap(d);
  a.partial = d.workspace;
  if (d.weight_grad) {
    a.ldb = d.ldb;
    a.ldc = d.k;
    a.N = (int)d.n;
    a.K = (int)d.k;
    a.tiles_n = (int)tiles_up(d.k, pl.bn);
    if (pl.kernel == Kernel::Big)
      return d.out_store == Store::F32 ? launch_big<float, TN>(a, s) : launch_big<__bf16, TN>(a, s);
    if (d.store == Store::F32) return launch_grouped<float, float, TN>(a, blocks, s);
    if (d.out_store == Store::F32) return launch_grouped<__bf16, float, TN>(a, blocks, s);
    return launch_grouped<__bf16, __bf16, TN>(a, blocks, s);
  }
  a.ldb = d.k;
  a.ldc = d.ldc;
  a.N = (int)(d.transpose_w ? d.k : d.n);
  a.K = (int)(d.transpose_w ? d.n : d.k);
  a.tiles_n = (int)tiles_up(a.N, pl.bn);
  if (!d.layer) return launch_rowwise(d, pl, a, blocks, s);
  layer.bias = d.bias;
  layer.R = d.R;
  layer.ldr = d.ldr;
  layer.Z = d.Z;
  layer.ldz = d.ldz;
  layer.act = d.act;
  layer.parts = split_parts(d);
  layer.part_tiles = (int)split_tiles(d);
  return launch_rowwise(d, pl, layer, blocks, s);
}

}  // namespace mns
