// A router's bookkeeping: the assignments of tokens to experts counted and put in the experts' order,
// and the balance loss with its gradient.
#include "mns_internal.h"

#include <type_traits>

namespace mns {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;

// ---- counts, offsets and order ------------------------------------------------------------------
//
// A stable counting sort of M assignments by expert (those of no expert last). Every block takes one
// piece of the list and every wave a part of that, both in order, so a place is: the expert's begin,
// plus what earlier blocks and waves hold of it, plus the rank inside the wave. With more than one
// block, a first launch counts each block's piece; the second adds the other blocks' counts by itself
// (four groups of threads side by side, E integers a block, from L2), scans them and deals the places. No
// atomics but counts in LDS, so the result is the one stable order. Bound by latency: few, long steps
// (524288 assignments of 256 experts, 8.4 MB: 3.6 + 13 us, of 32768 of 32 experts 2.9 + 4). Every block
// counting the whole list by itself, in one launch: 22.7 us for the latter.
struct OrderArgs {
  const int64_t* ids;
  int64_t* counts;
  int64_t* offsets;
  int64_t* order;              // may be null
  int* hist;                   // blocks x (E + 1)
  int M, E, blocks, piece;     // piece: assignments of a block, a multiple of the block's threads
};

__device__ __forceinline__ int bin_of(const OrderArgs& p, int i) {
  const int64_t id = p.ids[i];
  return id >= 0 && id < p.E ? (int)id : p.E;
}

__global__ __launch_bounds__(1024) void k_count(OrderArgs p) {
  __shared__ int bins[kMaxRouted + 1];
  for (int e = threadIdx.x; e <= p.E; e += 1024) bins[e] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * p.piece;
  const int end = (int)(first + p.piece < p.M ? first + p.piece : p.M);
#pragma unroll 4
  for (int i = (int)first + threadIdx.x; i < end; i += 1024) atomicAdd(&bins[bin_of(p, i)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += 1024)
    p.hist[(int64_t)blockIdx.x * (p.E + 1) + e] = bins[e];
}

// What some lanes of a wave wrote to LDS before is what its other lanes read behind it: the LDS takes a
// wave's accesses in order, and the compiler moves none across. No instruction.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// WAVES waves, whose counters for up to MOST experts fit the LDS: 16 for up to 512 (8192 assignments of 32
// experts in one block 9.0 us, with 4 waves 22.6), 4 beyond.
template <int WAVES, int MOST>
__global__ __launch_bounds__(64 * WAVES) void k_order(OrderArgs p) {
  constexpr int THREADS = 64 * WAVES, BINS = 256, SIDE = THREADS / BINS;
  static_assert(SIDE >= 1, "a thread for each bin of a step");
  __shared__ int cursor[WAVES][MOST + 1];     // counts, then the wave's next place, by expert
  __shared__ int sums[2][SIDE][BINS];         // of the blocks' counts: all, and those of earlier blocks
  __shared__ int carry[BINS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int bins = p.E + 1;
  for (int e = tid; e < bins * WAVES; e += THREADS) cursor[e / bins][e % bins] = 0;
  __syncthreads();
  const int share = p.piece / WAVES;
  const int64_t first = (int64_t)blockIdx.x * p.piece + (int64_t)wave * share;
  const int begin = (int)(first < p.M ? first : p.M);
  const int end = (int)(first + share < p.M ? first + share : p.M);
#pragma unroll 4
  for (int i = begin + lane; i < end; i += 64) atomicAdd(&cursor[wave][bin_of(p, i)], 1);
  // Bins in order, BINS at a time.
  int running = 0;
  for (int e0 = 0; e0 < bins; e0 += BINS) {
    const int e = e0 + tid % BINS, side = tid / BINS;
    if (p.blocks > 1) {
      int total = 0, before = 0;
      if (e < bins) {
#pragma unroll 8
        for (int b = side; b < p.blocks; b += SIDE) {
          const int h = p.hist[(int64_t)b * bins + e];
          total += h;
          before += b < (int)blockIdx.x ? h : 0;
        }
      }
      sums[0][side][tid % BINS] = total;
      sums[1][side][tid % BINS] = before;
    }
    __syncthreads();
    int total = 0, before = 0, own[WAVES], incl = 0;
    if (tid < BINS) {
      if (e < bins) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) total += own[w] = cursor[w][e];
        if (p.blocks > 1) {
          total = 0;
#pragma unroll
          for (int s = 0; s < SIDE; ++s) {
            total += sums[0][s][tid];
            before += sums[1][s][tid];
          }
        }
      }
      incl = total;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 63) carry[wave] = incl;
    }
    __syncthreads();
    int start = running + incl - total;
#pragma unroll
    for (int w = 0; w < BINS / 64; ++w) {
      if (w < wave) start += carry[w];
      running += carry[w];
    }
    if (tid < BINS && e < bins) {
      if (blockIdx.x == 0) {
        p.offsets[e] = start;
        if (e < p.E) p.counts[e] = total;
      }
      int place = start + before;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        cursor[w][e] = place;
        place += own[w];
      }
    }
    __syncthreads();
  }
  if (!p.order) return;
  int next = begin + lane < end ? bin_of(p, begin + lane) : -1;
  for (int i0 = begin; i0 < end; i0 += 64) {
    const int i = i0 + lane;
    const bool in = i < end;
    const int bin = next;
    next = i + 64 < end ? bin_of(p, i + 64) : -1;      // loaded a step ahead
    // the lanes of the same bin, one bit of the bin at a time
    unsigned long long same = __ballot(in);
    for (int bit = 1; bit < bins; bit <<= 1) {
      const unsigned long long set = __ballot((bin & bit) != 0);
      same &= (bin & bit) ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const int place = in ? cursor[wave][bin] : 0;
    wave_order();
    if (in) {
      p.order[place + rank] = i;
      if (rank == 0) cursor[wave][bin] = place + __popcll(same);
    }
    wave_order();
  }
}

// ---- the balance loss ------------------------------------------------------------------------------
//
// loss = scale E / N^2 sum_t a_t s_t with s_t = sum_e c_e p_te, p_t = softmax(logits_t); c_e: assignments
// of expert e, N: of all, a_t: of token t. Its gradient scale E / N^2 a_t p_te (c_e - s_t) needs a token's
// own row only, once the counts are known, so one pass reads the logits, adds up a_t s_t and writes the
// gradient: no sums over the tokens for each expert. G lanes hold a row, four neighbouring columns a
// lane and step; a row without an assignment is not looked at (whatever its logits hold). Bound by HBM
// where the batch is long (65536 tokens of 256 experts: 31 us, 4.4 TB/s of reads and writes), by latency
// below (16384 tokens of 32 experts in bfloat16, 2 MB: 4.5 us and 2 for the blocks' sums).
struct BalanceArgs {
  const void* logits; int64_t ld;
  const int64_t* ids;          // T x top
  const int64_t* counts;
  void* grad; int64_t ldg;     // may be null
  float* loss;
  double* partial;             // a block's sum of a_t s_t
  int T, E, top, blocks;
  float scale;
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, int valid, float (&v)[4], float rest) {
  T t[4];
  if (valid >= 4) {
    __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)t[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < valid ? (float)p[i] : rest;
  }
}

__device__ __forceinline__ void finish_loss(const BalanceArgs& p, double sum, double n) {
  *p.loss = n > 0. ? (float)((double)p.scale * p.E / (n * n) * sum) : 0.f;
}

// v op'ed over groups of G lanes, in each of them: up to 16 lanes by moves within the vector unit
// (neighbours, pairs, then the mirrored 8 and 16 lanes, whose halves are equal by then), beyond by
// shuffles, which go through LDS (65536 tokens of 256 experts, float32: 36.3 -> 30.9 us).
template <int G, typename V, typename F>
__device__ __forceinline__ V over_lanes(V v, F op) {
  static_assert(sizeof(V) == 4 && G >= 8, "one register");
  auto moved = [](V x, auto ctrl) {
    return __builtin_bit_cast(
        V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v = op(v, moved(v, std::integral_constant<int, 0xB1>{}));       // quad_perm [1, 0, 3, 2]
  v = op(v, moved(v, std::integral_constant<int, 0x4E>{}));       // quad_perm [2, 3, 0, 1]
  v = op(v, moved(v, std::integral_constant<int, 0x141>{}));      // row_half_mirror
  if constexpr (G >= 16) v = op(v, moved(v, std::integral_constant<int, 0x140>{}));   // row_mirror
  if constexpr (G >= 32) v = op(v, __shfl_xor(v, 16));
  if constexpr (G >= 64) v = op(v, __shfl_xor(v, 32));
  return v;
}

template <typename T, int G, int Q>
__global__ __launch_bounds__(kThreads) void k_balance(BalanceArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % G;
  constexpr int ROWS = 64 / G;                     // rows of a wave
  auto sum_of = [](auto v) { return over_lanes<G>(v, [](auto a, auto b) { return a + b; }); };
  double count[Q][4], n = 0., least = INFINITY;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = (q * G + l) * 4 + i;
      count[q][i] = e < p.E ? (double)p.counts[e] : 0.;
      n += count[q][i];
      if (e < p.E && count[q][i] < least) least = count[q][i];
    }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) {
    n += __shfl_xor(n, o, G);
    const double other = __shfl_xor(least, o, G);
    if (other < least) least = other;
  }
  // From here on by how much a count exceeds the least one: float32 keeps whole numbers up to 2^24 only, and
  // where the counts are larger but nearly equal, their differences are what the gradient is made of. No
  // term is negative, so what is added back for the loss takes nothing from its accuracy (counts less their
  // mean: a loss of probabilities on experts without assignments, 3e-7 of the mean, was 3e-3 of itself off).
  float c[Q][4];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[q][i] = (q * G + l) * 4 + i < p.E ? (float)(count[q][i] - least) : 0.f;
  const float factor = n > 0. ? (float)((double)p.scale * p.E / (n * n)) : 0.f;
  double total = 0.;
  for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * ROWS; t0 < p.T;
       t0 += (int64_t)p.blocks * kWaves * ROWS) {
    const int64_t t = t0 + lane / G;
    const bool in = t < p.T;
    int a = 0;
    for (int j = l; in && j < p.top; j += G) {
      const int64_t id = p.ids[t * p.top + j];
      a += id >= 0 && id < p.E;
    }
    a = sum_of(a);
    const bool use = in && a > 0;
    float x[Q][4], m = -INFINITY;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int col = (q * G + l) * 4;
      load4(static_cast<const T*>(p.logits) + t * p.ld + col, use ? p.E - col : 0, x[q], -INFINITY);
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, x[q][i]);
    }
    m = over_lanes<G>(m, [](float a, float b) { return fmaxf(a, b); });
    float z = 0.f, s = 0.f;
    // a row of lowest infinities has no probabilities: zeros (a NaN passes through the comparison)
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[q][i] = expf(x[q][i] - base);
        z += x[q][i];
        s += x[q][i] * c[q][i];
      }
    z = sum_of(z);
    s = sum_of(s);
    const float inv = z == 0.f ? 0.f : 1.f / z;
    s *= inv;
    // What s is off by, sum_e p_te (c_e - s): where one expert has nearly all of a token's probability, c_e - s
    // is as small as the rounding of s.
    float rest = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) rest += x[q][i] * (c[q][i] - s);
    rest = sum_of(rest) * inv;
    // (the s of a row without probabilities is nothing, not the least count)
    if (use && l == 0) total += (double)a * ((double)s + (double)rest + (z == 0.f ? 0. : least));
    if (p.grad && in) {
      const float f = use ? factor * (float)a * inv : 0.f;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int col = (q * G + l) * 4;
        T out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = (T)(use ? f * x[q][i] * (c[q][i] - s - rest) : 0.f);
        T* dst = static_cast<T*>(p.grad) + t * p.ldg + col;
        if (col + 4 <= p.E) {
          __builtin_memcpy(dst, out, sizeof(out));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + i < p.E) dst[i] = out[i];
        }
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  __shared__ double waves[kWaves];
  if (lane == 0) waves[wave] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) all += waves[w];
    if (p.blocks == 1) finish_loss(p, all, n);
    else p.partial[blockIdx.x] = all;
  }
}

__global__ __launch_bounds__(kThreads) void k_balance_join(BalanceArgs p) {
  const int tid = threadIdx.x;
  double sum = 0., n = 0.;
#pragma unroll 4
  for (int b = tid; b < p.blocks; b += kThreads) sum += p.partial[b];
  for (int e = tid; e < p.E; e += kThreads) n += (double)p.counts[e];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    sum += __shfl_xor(sum, o);
    n += __shfl_xor(n, o);
  }
  __shared__ double s[2][kWaves];
  if ((tid & 63) == 0) {
    s[0][tid >> 6] = sum;
    s[1][tid >> 6] = n;
  }
  __syncthreads();
  if (tid != 0) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    sum += s[0][w];
    n += s[1][w];
  }
  finish_loss(p, sum, n);
}

// One block and launch up to kOneBlock assignments (4096 of 32 or 256 experts: 6.0, 8.1 us; in two launches
// 6.7, 8.6; 8192: 9.0, 11.8 against 7.0, 8.8). Beyond, pieces of 1024 to 64 blocks (32768: 6.7, 8.9 us;
// pieces of 2048 8.0, 10.2), of 2048 to 128 (131072: 7.9, 10.8; of 1024 8.1, 11.8, of 4096 9.1, 11.8), then
// 128 larger ones, as every block adds all the blocks' counts.
constexpr int64_t kOneBlock = 4096;
int order_blocks(int64_t m, int* piece) {
  const int64_t c = m <= kOneBlock ? (m + 1023) / 1024 * 1024 : m <= 64 * 1024 ? 1024 : m <= 128 * 2048 ? 2048
                                               : (m + 128 * 1024 - 1) / (128 * 1024) * 1024;
  *piece = (int)(c < 1024 ? 1024 : c);
  return m <= kOneBlock ? 1 : (int)((m + c - 1) / c);
}

// (65536 tokens of 256 experts, float32, 134 MB: 30.4 us; 512 blocks took 1.8 times as long, 8192 blocks 1.25)
constexpr int kBalanceBlocks = 2048;

template <typename T>
hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.blocks), block(kThreads);
  if (a.E <= 32) hipLaunchKernelGGL((k_balance<T, 8, 1>), grid, block, 0, s, a);
  else if (a.E <= 64) hipLaunchKernelGGL((k_balance<T, 16, 1>), grid, block, 0, s, a);
  else if (a.E <= 128) hipLaunchKernelGGL((k_balance<T, 32, 1>), grid, block, 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_balance<T, 64, 1>), grid, block, 0, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL((k_balance<T, 64, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_balance<T, 64, kMaxRouted / 256>), grid, block, 0, s, a);
  return hipGetLastError();
}

int balance_blocks(int64_t tokens, int64_t experts) {
  const int64_t lanes = experts <= 32 ? 8 : experts <= 64 ? 16 : experts <= 128 ? 32 : 64;
  const int64_t rows = kWaves * 64 / lanes, blocks = (tokens + rows - 1) / rows;
  // two rounds of one block take less than a second launch (64 tokens of 32 experts: 4.3 against 5.5 us),
  // four do not (128 tokens: 6.1 against 5.5; 16 of 256 experts: 7.5 against 5.9)
  if (blocks <= 2) return 1;
  return (int)(blocks < 1 ? 1 : blocks > kBalanceBlocks ? kBalanceBlocks : blocks);
}

}  // namespace

size_t order_workspace(int64_t assignments, int64_t experts) {
  int piece;
  const int blocks = order_blocks(assignments, &piece);
  return blocks > 1 ? (size_t)blocks * (experts + 1) * sizeof(int) : 0;
}

hipError_t expert_order(const int64_t* ids, int64_t assignments, int64_t experts, int64_t* counts,
                        int64_t* offsets, int64_t* order, void* workspace, hipStream_t s) {
  OrderArgs a;
  a.ids = ids;
  a.counts = counts;
  a.offsets = offsets;
  a.order = order;
  a.hist = static_cast<int*>(workspace);
  a.M = (int)assignments;
  a.E = (int)experts;
  a.blocks = order_blocks(assignments, &a.piece);
  if (a.blocks > 1) {
    hipLaunchKernelGGL(k_count, dim3((unsigned)a.blocks), dim3(1024), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)a.blocks);
  if (experts <= 512) hipLaunchKernelGGL((k_order<16, 512>), grid, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((k_order<4, kMaxRouted>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

size_t balance_workspace(int64_t tokens, int64_t experts) {
  const int b = balance_blocks(tokens, experts);
  return b > 1 ? (size_t)b * sizeof(double) : 0;
}

hipError_t balance(const BalanceDesc& d, hipStream_t s) {
  BalanceArgs a;
  a.logits = d.logits;
  a.ld = d.ld;
  a.ids = d.ids;
  a.counts = d.counts;
  a.grad = d.grad;
  a.ldg = d.ldg;
  a.loss = d.loss;
  a.partial = static_cast<double*>(d.workspace);
  a.T = (int)d.tokens;
  a.E = (int)d.experts;
  a.top = (int)d.top;
  a.blocks = balance_blocks(d.tokens, d.experts);
  a.scale = d.scale;
  const hipError_t e = d.store == Store::F32 ? launch_balance<float>(a, s)
                                             : launch_balance<__bf16>(a, s);
  if (e != hipSuccess || a.blocks == 1) return e;
  hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace mns
