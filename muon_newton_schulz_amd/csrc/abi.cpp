// C ABI of the Muon / Newton-Schulz step: argument validation, workspace planning and the
// drivers that sequence the kernels of one step on the caller's stream.
//
// Method: page "Dion3: Full-stack orthogonal updates" -- Eq. (1) (Muon), Eq. (2) (NorMuon),
// section "Standard Newton-Schulz", Theorem 2 and the restart of Algorithm 3 (Gram NS),
// Algorithm 4 (Dion3 row selection), section "4. Megabatched Communication" (matrices of
// one shape are processed as one batch).
#include "muon_ns.h"
#include "activation.h"
#include "mns_internal.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

using namespace mns;

namespace {

// ---- instrumentation: hipEvent pairs around every launch while a session is open ----------

struct ProfRec {
  const char* name;
  hipEvent_t a, b;
  double flops, bytes;
};
// g_prof_on is read on every launch without the lock (atomic: a session toggled on another
// thread is seen cleanly); the record list and the failure flag are guarded by g_prof_mu.
std::mutex g_prof_mu;
std::atomic<bool> g_prof_on{false};
bool g_prof_failed = false;
std::vector<ProfRec> g_prof;
// Optional cache flush before the session's HBM-bound launches (mns_profile_set_flush).
void* g_flush_buf = nullptr;
size_t g_flush_bytes = 0;
constexpr double kFlushMinBytes = double(16 << 20);

template <typename F>
hipError_t timed(const char* name, double flops, double bytes, hipStream_t s, F&& launch) {
  if (!g_prof_on.load(std::memory_order_acquire)) return launch();
  {
    void* fb = nullptr;
    size_t fn = 0;
    {
      std::lock_guard<std::mutex> lk(g_prof_mu);
      fb = g_flush_buf;
      fn = g_flush_bytes;
    }
    // outside the event pair: the launch then reads its operands from HBM
    if (fb && fn && flops == 0.0 && bytes >= kFlushMinBytes) {
      const hipError_t fe = cache_flush(fb, fn, s);
      if (fe != hipSuccess) return fe;
    }
  }
  ProfRec r{name, nullptr, nullptr, flops, bytes};
  if (hipEventCreate(&r.a) != hipSuccess || hipEventCreate(&r.b) != hipSuccess) {
    if (r.a) (void)hipEventDestroy(r.a);   // the first event was made, the second was not
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_prof_failed = true;
    return launch();
  }
  (void)hipEventRecord(r.a, s);
  const hipError_t e = launch();
  (void)hipEventRecord(r.b, s);
  std::lock_guard<std::mutex> lk(g_prof_mu);
  try {
    g_prof.push_back(r);
  } catch (...) {                          // no host memory: the session fails, the call does not
    (void)hipEventDestroy(r.a);
    (void)hipEventDestroy(r.b);
    g_prof_failed = true;
  }
  return e;
}

hipError_t timed_gemm(const GemmDesc& d, double flops, hipStream_t s) {
  return timed(gemm_name(d), flops, 0.0, s, [&] { return gemm(d, s); });
}



constexpr int64_t kMaxDim = 65536;
constexpr int64_t kMaxElems = 2147483647LL;
constexpr int kMaxT = 64;
constexpr int kChunk = kMaxPack;      // matrices per batched launch sequence

// Carves 256-byte aligned slices from the workspace; with a null base it only measures.
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename T>
  T* take(size_t count) {
    off = (off + 255) & ~size_t(255);
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += count * sizeof(T);
    return p;
  }
};

// Geometry of the Newton-Schulz problem for a rows x cols matrix: it runs on the short
// side (n <= m), a tall matrix through its transpose, in a zero-padded n_p x m_p iterate
// whose entries are stored times S (a power of two chosen so the float16 iterate keeps
// its entries well inside the normal range: X_0 entries ~ S/sqrt(nm), later ~ S/sqrt(m)).
struct Geo {
  int64_t rows, cols, n, m, n_p, m_p;
  int64_t rows_p, cols_p;      // stored layout, padded (the result O is kept this way)
  int64_t ld_x, ld_t, ld_q;    // row pitch of X (n_p x m_p), X^T (m_p x n_p), n_p x n_p
  bool tall;
  Elem elem;
  float S;
};

Geo make_geo(int64_t rows, int64_t cols, Store st) {
  Geo g;
  g.rows = rows;
  g.cols = cols;
  g.tall = rows > cols;
  g.n = g.tall ? cols : rows;
  g.m = g.tall ? rows : cols;
  g.n_p = pad_up(g.n);
  g.m_p = pad_up(g.m);
  g.rows_p = pad_up(rows);
  g.cols_p = pad_up(cols);
  g.ld_x = padded_ld(g.m_p);
  g.ld_t = padded_ld(g.n_p);
  g.ld_q = padded_ld(g.n_p);
  g.elem = st == Store::BF16 ? Elem::F16 : Elem::F32;
  if (g.elem == Elem::F16) {
    int e = (int)std::lround(0.5 * std::log2((double)g.m));
    if (e < 0) e = 0;
    if (e > 12) e = 12;
    g.S = std::ldexp(1.0f, e);
  } else {
    g.S = 1.0f;
  }
  return g;
}

// The iterate X (n_p x m_p, rows = the short side) feeds X X^T and, read k-major, B X and
// Q X; its transposed copy X^T (m_p x n_p) is formed only where those products cannot read X
// k-major (64 x 64 tiles, float32) and as the stored layout of a tall result. Each layout
// has a ping-pong pair.
struct NsBuffers {
  void* X[2] = {};
  void* Xt[2] = {};
  void* sq[6] = {};        // n_p x n_p scratch: standard uses 2, Gram uses 6
  float* gemm_scratch = nullptr;
  size_t gemm_scratch_bytes = 0;
  int64_t x_stride = 0, xt_stride = 0, sq_stride = 0;   // batch strides (elements)
};

// Split-k scratch the GEMMs of this geometry can use at most: (output tiles) x (k-tiles / 8)
// float32 tiles (before any cap).
size_t gemm_scratch_need(const Geo& g, int count) {
  const size_t kparts = (size_t)(g.m_p > g.n_p ? g.m_p : g.n_p) / 256;
  return (size_t)count * g.n_p * g.n_p * kparts * sizeof(float);
}

void carve_ns(Carver& cv, const Geo& g, int count, int kind, NsBuffers& b,
              size_t gemm_cap = kGemmScratchBytes) {
  const size_t es = (size_t)elem_bytes(g.elem);
  b.x_stride = g.n_p * g.ld_x;
  b.xt_stride = g.m_p * g.ld_t;
  b.sq_stride = g.n_p * g.ld_q;
  for (int i = 0; i < 2; ++i) {
    b.X[i] = cv.take<char>(es * count * b.x_stride);
    b.Xt[i] = cv.take<char>(es * count * b.xt_stride);
  }
  const int nsq = kind == MNS_NS_GRAM ? 6 : 2;
  for (int i = 0; i < nsq; ++i) b.sq[i] = cv.take<char>(es * count * b.sq_stride);
  // split-k partial sums: at most (output tiles) x (k-tiles / 8) tiles of float32, capped (a
  // smaller cap only makes the GEMMs split their tail tiles into fewer parts)
  size_t scratch = gemm_scratch_need(g, count);
  if (scratch > gemm_cap) scratch = gemm_cap;
  b.gemm_scratch = cv.take<float>(scratch / sizeof(float));
  b.gemm_scratch_bytes = scratch;
}

// Normalisation targets: the stored layout of the source is X for a wide matrix and X^T for
// a tall one; the other buffer receives the transpose.
// With km (the products read X k-major) only X is formed: null for the X^T side.
void* straight(const Geo& g, const NsBuffers& b, bool km) {
  return g.tall ? (km ? nullptr : b.Xt[0]) : b.X[0];
}
void* transposed(const Geo& g, const NsBuffers& b, bool km) {
  return g.tall ? b.X[0] : (km ? nullptr : b.Xt[0]);
}

#define MNS_HIP(expr)                               \
  do {                                              \
    if ((expr) != hipSuccess) return MNS_ERR_HIP;   \
  } while (0)

GemmDesc sym_desc(const Geo& g, int count, const NsBuffers& b, const void* A, const void* B,
                  int64_t ldab, int64_t sab, int K, void* C) {
  GemmDesc d;
  d.elem = g.elem;
  d.A = A; d.lda = ldab; d.sA = sab;
  d.B = B; d.ldb = ldab; d.sB = sab;
  d.C = C; d.ldc = g.ld_q; d.sC = b.sq_stride;
  d.M = (int)g.n_p; d.N = (int)g.n_p; d.K = K; d.batch = count;
  d.sym = true;
  d.partial = b.gemm_scratch; d.partial_bytes = b.gemm_scratch_bytes;
  return d;
}

// L X for L n_p x n_p (symmetric) and X given by its transpose Xt (m_p x n_p): written to
// C (n_p x m_p) and/or Ct (m_p x n_p).
GemmDesc left_desc(const Geo& g, int count, const NsBuffers& b, const void* L, const void* Xt,
                   void* C, void* Ct) {
  GemmDesc d;
  d.elem = g.elem;
  d.A = L; d.lda = g.ld_q; d.sA = b.sq_stride;
  d.B = Xt; d.ldb = g.ld_t; d.sB = b.xt_stride;
  d.C = C; d.ldc = g.ld_x; d.sC = b.x_stride;
  d.Ct = Ct; d.ldct = g.ld_t; d.sCt = b.xt_stride;
  d.M = (int)g.n_p; d.N = (int)g.m_p; d.K = (int)g.n_p; d.batch = count;
  d.partial = b.gemm_scratch; d.partial_bytes = b.gemm_scratch_bytes;
  return d;
}

// Whether the products L X of this geometry read the iterate X itself, k-major (float16 on
// 256 x 256 or 128 x 128 tiles): X^T is then never formed, except as the stored layout of a
// tall result.
bool kmajor_ns(const Geo& g, int count, const NsBuffers& b) {
  return gemm_kmajor_ok(left_desc(g, count, b, nullptr, nullptr, b.X[1], nullptr));
}

// L X for the iterate X[cur] (through X^T[cur], or k-major from X[cur] when km).
GemmDesc lx_desc(const Geo& g, int count, const NsBuffers& b, bool km, const void* L, int cur,
                 void* C, void* Ct) {
  GemmDesc d = left_desc(g, count, b, L, b.Xt[cur], C, Ct);
  if (km) {
    d.B = b.X[cur]; d.ldb = g.ld_x; d.sB = b.x_stride;
    d.b_kmajor = true;
  }
  return d;
}

// Optional request for the per-row sums of squares of the NS result (NorMuon's row
// statistics), taken in the epilogue of the product that writes the result: part gets the
// GemmDesc::rowsq layout (64-column chunks); done reports whether such a product ran.
struct RowSq {
  float* part = nullptr;
  int rows = 0;
  bool done = false;
};

void want_rowsq(GemmDesc& d, RowSq* rs) {
  if (!rs) return;
  d.rowsq = rs->part;
  d.rowsq_rows = rs->rows;
  rs->done = true;
}

// Standard quintic NS on the normalised iterate (b.X[0], b.Xt[0]) (section "Standard
// Newton-Schulz"): A = X X^T, B = b A + c A^2, X <- a X + B X. Returns the result in the
// stored layout (X for a wide matrix, X^T for a tall one; row pitch padded_ld(cols_p)).
mns_status run_standard(const Geo& g, int count, const NsBuffers& b, int T, const float* abc,
                        hipStream_t s, void** out, RowSq* rs) {
  int cur = 0;
  void* A = b.sq[0];
  void* B = b.sq[1];
  const float inv_s2 = 1.0f / (g.S * g.S);
  const double nn = (double)count * g.n * g.n;
  const bool km = kmajor_ns(g, count, b);
  for (int t = 0; t < T; ++t) {
    const float a = abc[3 * t], bb = abc[3 * t + 1], c = abc[3 * t + 2];
    GemmDesc gram = sym_desc(g, count, b, b.X[cur], b.X[cur], g.ld_x, b.x_stride, (int)g.m_p, A);
    gram.alpha = inv_s2;
    MNS_HIP(timed_gemm(gram, nn * g.m, s));
    const bool last = t == T - 1;
    // X is needed for the next X X^T (and, k-major, the next update); X^T only for the next
    // update when it cannot read X k-major, and as the stored layout of a tall result.
    GemmDesc upd = lx_desc(g, count, b, km, A, cur, (!last || !g.tall) ? b.X[cur ^ 1] : nullptr,
                           (last ? g.tall : !km) ? b.Xt[cur ^ 1] : nullptr);
    if (c != 0.0f) {
      // P = a I + b A + c A^2 (a on the real diagonal only, so padding stays zero), then
      // X <- P X: the same map as a X + (b A + c A^2) X, without re-reading X.
      GemmDesc poly = sym_desc(g, count, b, A, A, g.ld_q, b.sq_stride, (int)g.n_p, B);
      poly.alpha = c;
      poly.beta = bb;
      poly.D = A; poly.ldd = g.ld_q; poly.sD = b.sq_stride;
      poly.gamma = a;
      poly.diag_limit = (int)g.n;
      MNS_HIP(timed_gemm(poly, nn * g.n, s));
      upd.A = B;
    } else {
      upd.alpha = bb;
      upd.beta = a;
      upd.D = b.X[cur]; upd.ldd = g.ld_x; upd.sD = b.x_stride;   // read in C coordinates
    }
    if (last) want_rowsq(upd, rs);
    MNS_HIP(timed_gemm(upd, 2.0 * nn * g.m, s));
    cur ^= 1;
  }
  *out = g.tall ? b.Xt[cur] : b.X[cur];
  return MNS_OK;
}

// Gram Newton-Schulz (Theorem 2) with restarts (Algorithm 3): R = X X^T; per iteration
// Z = a I + b R + c R^2, R <- R Z^2 (skipped when unused), Q <- Q Z (Q_1 = Z_1);
// a restart before t forms X <- Q X, R <- X X^T, Q <- I. Output Q X (stored layout).
// Whether restart_mask asks for a restart before iteration t (bits 2..31; a 32-bit mask
// cannot name a later iteration, and a shift by 32 or more would be undefined).
inline bool restart_at(uint32_t restart_mask, int t) {
  return t >= 0 && t < 32 && ((restart_mask >> t) & 1u);
}

mns_status run_gram(const Geo& g, int count, const NsBuffers& b, int T, const float* abc,
                    uint32_t restart_mask, hipStream_t s, void** out, RowSq* rs) {
  int cur = 0;
  void* R = b.sq[0];
  void* Rt = b.sq[1];
  void* Z = b.sq[2];
  void* Z2 = b.sq[3];
  void* Q = b.sq[4];
  void* Qt = b.sq[5];
  const float inv_s2 = 1.0f / (g.S * g.S);
  const int n = (int)g.n_p;
  const double nn = (double)count * g.n * g.n;
  const bool km = kmajor_ns(g, count, b);

  GemmDesc gram = sym_desc(g, count, b, b.X[cur], b.X[cur], g.ld_x, b.x_stride, (int)g.m_p, R);
  gram.alpha = inv_s2;
  MNS_HIP(timed_gemm(gram, nn * g.m, s));
  bool q_identity = true;
  for (int t = 1; t <= T; ++t) {
    const float a = abc[3 * (t - 1)], bb = abc[3 * (t - 1) + 1], c = abc[3 * (t - 1) + 2];
    if (t > 1 && restart_at(restart_mask, t)) {
      if (!q_identity) {
        MNS_HIP(timed_gemm(lx_desc(g, count, b, km, Q, cur, b.X[cur ^ 1],
                                   km ? nullptr : b.Xt[cur ^ 1]),
                           2.0 * nn * g.m, s));
        cur ^= 1;
      }
      GemmDesc re = sym_desc(g, count, b, b.X[cur], b.X[cur], g.ld_x, b.x_stride, (int)g.m_p, R);
      re.alpha = inv_s2;
      MNS_HIP(timed_gemm(re, nn * g.m, s));
      q_identity = true;
    }
    GemmDesc zd = sym_desc(g, count, b, R, R, g.ld_q, b.sq_stride, n, Z);
    zd.alpha = c;
    zd.beta = bb;
    zd.D = R; zd.ldd = g.ld_q; zd.sD = b.sq_stride;
    zd.gamma = a;
    zd.diag_limit = (int)g.n;
    MNS_HIP(timed_gemm(zd, nn * g.n, s));
    if (t < T && !restart_at(restart_mask, t + 1)) {
      MNS_HIP(timed_gemm(sym_desc(g, count, b, Z, Z, g.ld_q, b.sq_stride, n, Z2), nn * g.n, s));
      MNS_HIP(timed_gemm(sym_desc(g, count, b, R, Z2, g.ld_q, b.sq_stride, n, Rt), nn * g.n, s));
      void* tmp = R; R = Rt; Rt = tmp;
    }
    if (q_identity) {
      void* tmp = Q; Q = Z; Z = tmp;
      q_identity = false;
    } else {
      MNS_HIP(timed_gemm(sym_desc(g, count, b, Q, Z, g.ld_q, b.sq_stride, n, Qt), nn * g.n, s));
      void* tmp = Q; Q = Qt; Qt = tmp;
    }
  }
  if (q_identity) {
    *out = g.tall ? b.Xt[cur] : b.X[cur];
  } else {
    GemmDesc fin = lx_desc(g, count, b, km, Q, cur, g.tall ? nullptr : b.X[cur ^ 1],
                           g.tall ? b.Xt[cur ^ 1] : nullptr);
    want_rowsq(fin, rs);
    MNS_HIP(timed_gemm(fin, 2.0 * nn * g.m, s));
    *out = g.tall ? b.Xt[cur ^ 1] : b.X[cur ^ 1];
  }
  return MNS_OK;
}

mns_status run_ns(const Geo& g, int count, const NsBuffers& b, int kind, int T, const float* abc,
                  uint32_t restart_mask, hipStream_t s, void** out, RowSq* rs = nullptr) {
  if (kind == MNS_NS_GRAM) return run_gram(g, count, b, T, abc, restart_mask, s, out, rs);
  return run_standard(g, count, b, T, abc, s, out, rs);
}

// ---- validation helpers --------------------------------------------------------------------

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

mns_status check_shape(int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 1 || rows < 1 || cols < 1) return MNS_ERR_SHAPE;
  if (rows > kMaxDim || cols > kMaxDim || rows * cols > kMaxElems) return MNS_ERR_SHAPE;
  if (batch > kMaxElems / (rows * cols)) return MNS_ERR_SHAPE;
  return MNS_OK;
}

// The GEMMs address one padded iterate (either layout, with its row pitch) with 32-bit byte
// offsets.
mns_status check_iterate(int64_t rows, int64_t cols, Store st) {
  const int64_t rp = pad_up(rows), cp = pad_up(cols);
  const int64_t a = rp * padded_ld(cp), b = cp * padded_ld(rp);
  const int64_t bytes = (a > b ? a : b) * (st == Store::BF16 ? 2 : 4);
  return bytes <= kMaxElems ? MNS_OK : MNS_ERR_SHAPE;
}

mns_status check_dtype(int dt) {
  return (dt == MNS_F32 || dt == MNS_BF16) ? MNS_OK : MNS_ERR_DTYPE;
}

mns_status check_ns(int T, const float* abc, int kind, uint32_t restart_mask) {
  if (T < 1 || T > kMaxT) return MNS_ERR_PARAM;
  if (!abc) return MNS_ERR_NULL;
  for (int i = 0; i < 3 * T; ++i)
    if (!std::isfinite(abc[i])) return MNS_ERR_PARAM;
  if (kind != MNS_NS_STANDARD && kind != MNS_NS_GRAM) return MNS_ERR_PARAM;
  if (kind == MNS_NS_STANDARD && restart_mask != 0) return MNS_ERR_PARAM;
  // valid restart bits: 2..T
  const uint64_t allowed = ((T >= 31 ? 0xFFFFFFFFull : ((1ull << (T + 1)) - 1))) & ~3ull;
  if ((uint64_t)restart_mask & ~allowed) return MNS_ERR_PARAM;
  return MNS_OK;
}

mns_status check_ws(void* ws, size_t have, size_t need) {
  if (!ws) return MNS_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MNS_ERR_WORKSPACE;
  if (have < need) return MNS_ERR_WORKSPACE;
  return MNS_OK;
}

int64_t k_rows(double f, int64_t rows) {
  int64_t k = (int64_t)std::ceil(f * (double)rows);
  if (k < 1) k = 1;
  if (k > rows) k = rows;
  return k;
}

// Shape groups: matrices of equal (rows, cols), in order of first appearance. False where the host has no
// memory for them.
struct Group {
  int64_t rows, cols;
  std::vector<int> idx;
};

bool group_by_shape(const mns_matrix* mats, int count, std::vector<Group>& gs) try {
  for (int i = 0; i < count; ++i) {
    bool found = false;
    for (auto& g : gs)
      if (g.rows == mats[i].rows && g.cols == mats[i].cols) {
        g.idx.push_back(i);
        found = true;
        break;
      }
    if (!found) gs.push_back(Group{mats[i].rows, mats[i].cols, {i}});
  }
  return true;
} catch (...) {
  return false;
}

mns_status validate_step(const mns_matrix* mats, int count, const mns_hparams* hp,
                         bool need_ptrs) {
  if (!mats || !hp) return MNS_ERR_NULL;
  if (count < 1) return MNS_ERR_SHAPE;
  mns_status st = check_dtype(hp->dtype);
  if (st != MNS_OK) return st;
  st = check_ns(hp->T, hp->abc, hp->kind, hp->restart_mask);
  if (st != MNS_OK) return st;
  if (!std::isfinite(hp->mu) || !std::isfinite(hp->lr)) return MNS_ERR_PARAM;
  if (!(hp->row_fraction > 0.0 && hp->row_fraction <= 1.0)) return MNS_ERR_PARAM;
  if (hp->normuon != 0 && hp->normuon != 1) return MNS_ERR_PARAM;
  if (hp->normuon && (!(hp->beta2 >= 0.f && hp->beta2 <= 1.f) || !(hp->eps >= 0.f) ||
                      !std::isfinite(hp->eps)))
    return MNS_ERR_PARAM;
  for (int i = 0; i < count; ++i) {
    st = check_shape(1, mats[i].rows, mats[i].cols);
    if (st != MNS_OK) return st;
    st = check_iterate(mats[i].rows, mats[i].cols, hp->dtype == MNS_BF16 ? Store::BF16 : Store::F32);
    if (st != MNS_OK) return st;
    if (need_ptrs) {
      if (!mats[i].W || !mats[i].M || !mats[i].G) return MNS_ERR_NULL;
      if (hp->normuon && !mats[i].v) return MNS_ERR_NULL;
      if (!aligned(mats[i].W, 16) || !aligned(mats[i].M, 16) || !aligned(mats[i].G, 16) ||
          (mats[i].v && !aligned(mats[i].v, 4)))
        return MNS_ERR_PARAM;
    }
  }
  return MNS_OK;
}

// Workspace layout of one chunk (<= kChunk matrices of one shape) of muon_step.
struct StepWs {
  double* partials = nullptr;
  float* xscale = nullptr;
  NsBuffers ns;
  float* part = nullptr;
  float* rowscale = nullptr;
  double* fin = nullptr;
  float* l1 = nullptr;
  double* l2sq = nullptr;
  int32_t* S = nullptr;
  int nblk = 0, chunks = 0;
};

size_t carve_step(void* base, const Geo& g, int count, int64_t rows, int64_t cols, bool dion,
                  int64_t k, int kind, StepWs& w) {
  Carver cv(base);
  w.nblk = dion ? 0 : norm_blocks(rows * cols);
  w.partials = cv.take<double>((size_t)count * w.nblk);
  w.xscale = cv.take<float>((size_t)count);
  carve_ns(cv, g, count, kind, w.ns);
  w.chunks = (int)(g.cols_p / 64);                     // row-norm partials per stored row
  w.part = cv.take<float>((size_t)count * w.chunks * g.rows);
  w.rowscale = cv.take<float>((size_t)count * g.rows);
  w.fin = cv.take<double>((size_t)count * 2 * normuon_blocks(g.rows));
  if (dion) {
    w.l1 = cv.take<float>((size_t)count * rows);
    w.S = cv.take<int32_t>((size_t)count * k);
    w.l2sq = cv.take<double>((size_t)count * rows);
  }
  return cv.off + 256;
}

size_t step_bytes(const std::vector<Group>& groups, const mns_hparams* hp) {
  const Store st = hp->dtype == MNS_BF16 ? Store::BF16 : Store::F32;
  const bool dion = hp->row_fraction < 1.0;
  size_t need = 0;
  for (const Group& gr : groups) {
    const int c = (int)gr.idx.size() < kChunk ? (int)gr.idx.size() : kChunk;
    const int64_t k = dion ? k_rows(hp->row_fraction, gr.rows) : gr.rows;
    const Geo g = make_geo(k, gr.cols, st);
    StepWs w;
    const size_t b = carve_step(nullptr, g, c, gr.rows, gr.cols, dion, k, hp->kind, w);
    if (b > need) need = b;
  }
  return need;
}

// One chunk of c matrices of one shape: the momentum and its norm, the Newton-Schulz iterations on
// g (k x cols) and the weight update. With Gp null the momentum already holds its new values,
// the c matrices of M consecutive from M_base (never with Dion3's row selection).
mns_status step_chunk(const Geo& g, int c, int64_t rows, int64_t cols, int64_t k,
                      const mns_hparams* hp, const PtrPack& Wp, const PtrPack& Mp,
                      const PtrPack* Gp, const float* M_base, const PtrPack& Vp, void* workspace,
                      hipStream_t s) {
  const Store sto = hp->dtype == MNS_BF16 ? Store::BF16 : Store::F32;
  const bool dion = hp->row_fraction < 1.0;
  StepWs w;
  carve_step(workspace, g, c, rows, cols, dion, k, hp->kind, w);
  const bool km = kmajor_ns(g, c, w.ns);

  const double all = (double)c * rows * cols;      // elements of the chunk's matrices
  const double sel = (double)c * k * cols;         // elements the NS runs on
  const double es = elem_bytes(g.elem), ss = sto == Store::BF16 ? 2.0 : 4.0;
  if (!dion) {
    if (Gp) {
      MNS_HIP(timed("momentum", 0, all * (8.0 + ss), s, [&] {
        return momentum(Mp, *Gp, sto, c, rows * cols, hp->mu, w.partials, s); }));
    } else {
      MNS_HIP(timed("sumsq", 0, all * 4.0, s, [&] {
        return sumsq(M_base, Store::F32, c, rows * cols, w.partials, s); }));
    }
    MNS_HIP(timed("finalize_scale", 0, 4.0 * c * w.nblk, s, [&] {
      return finalize_scale(w.partials, w.nblk, c, g.S, w.xscale, s); }));
    MNS_HIP(timed("normalize", 0, all * (4.0 + (km ? 1.0 : 2.0) * es), s, [&] {
      return normalize(&Mp, nullptr, true, sto, c, rows, cols, w.xscale, g.elem,
                       straight(g, w.ns, km), transposed(g, w.ns, km), g.rows_p,
                       g.cols_p, s); }));
  } else {
    MNS_HIP(timed("momentum_l1", 0, all * (8.0 + ss), s, [&] {
      return momentum_l1(Mp, *Gp, sto, c, rows, cols, w.l1, w.l2sq, s); }));
    MNS_HIP(timed("topk", 0, 8.0 * c * rows + 8.0 * c * k, s, [&] {
      return topk_rows(w.l1, w.l2sq, c, rows, k, g.S, w.S, w.xscale, s); }));
    MNS_HIP(timed("gather_normalize", 0, sel * (8.0 + (km ? 1.0 : 2.0) * es), s, [&] {
      return gather_normalize(Mp, c, k, cols, w.S, hp->mu, w.xscale, g.elem,
                              straight(g, w.ns, km), transposed(g, w.ns, km), g.rows_p,
                       g.cols_p, s); }));
  }
  void* O = nullptr;
  RowSq rs;
  rs.part = w.part;
  rs.rows = (int)k;
  const mns_status st = run_ns(g, c, w.ns, hp->kind, hp->T, hp->abc, hp->restart_mask, s, &O,
              hp->normuon ? &rs : nullptr);
  if (st != MNS_OK) return st;
  const float inv_s = 1.0f / g.S;
  if (hp->normuon) {
    // The row statistics come from the epilogue of the product that wrote the result
    // (every run ends with one: T >= 1).
    if (!rs.done) return MNS_ERR_PARAM;
    MNS_HIP(timed("normuon_finalize", 0, 4.0 * c * k * (w.chunks + 3), s, [&] {
      return normuon_finalize(w.part, w.chunks, c, k, cols, &Vp, nullptr, 0,
                              dion ? w.S : nullptr, hp->beta2, hp->eps, inv_s * inv_s, inv_s,
                              w.rowscale, w.fin, s); }));
  } else {
    MNS_HIP(timed("fill", 0, 4.0 * c * k, s, [&] {
      return fill(w.rowscale, (int64_t)c * k, inv_s, s); }));
  }
  MNS_HIP(timed("weight_update", 0, sel * (2.0 * ss + es) + 4.0 * c * k, s, [&] {
    return weight_update(Wp, sto, c, k, cols, O, g.elem, g.rows_p, g.cols_p, w.rowscale,
                         dion ? w.S : nullptr, k, hp->lr, s); }));
  return MNS_OK;
}

}  // namespace

extern "C" {

const char* mns_status_string(int status) {
  switch (status) {
    case MNS_OK: return "MNS_OK";
    case MNS_ERR_NULL: return "MNS_ERR_NULL: a required pointer is NULL";
    case MNS_ERR_SHAPE: return "MNS_ERR_SHAPE: a size is out of range";
    case MNS_ERR_DTYPE: return "MNS_ERR_DTYPE: unknown storage dtype";
    case MNS_ERR_PARAM: return "MNS_ERR_PARAM: invalid hyperparameter or alignment";
    case MNS_ERR_WORKSPACE: return "MNS_ERR_WORKSPACE: workspace NULL, misaligned or too small";
    case MNS_ERR_HIP: return "MNS_ERR_HIP: a HIP launch failed";
    default: return "unknown mns_status";
  }
}

int mns_version(void) { return 100; }

mns_status mns_step_workspace_size(const mns_matrix* mats, int count, const mns_hparams* hp,
                                   size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  const mns_status st = validate_step(mats, count, hp, false);
  if (st != MNS_OK) return st;
  std::vector<Group> groups;
  if (!group_by_shape(mats, count, groups)) return MNS_ERR_PARAM;
  *bytes = step_bytes(groups, hp);
  return MNS_OK;
}

mns_status muon_step(const mns_matrix* mats, int count, const mns_hparams* hp, void* workspace,
                     size_t workspace_bytes, void* stream) {
  mns_status st = validate_step(mats, count, hp, true);
  if (st != MNS_OK) return st;
  std::vector<Group> groups;
  if (!group_by_shape(mats, count, groups)) return MNS_ERR_PARAM;
  st = check_ws(workspace, workspace_bytes, step_bytes(groups, hp));
  if (st != MNS_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Store sto = hp->dtype == MNS_BF16 ? Store::BF16 : Store::F32;
  const bool dion = hp->row_fraction < 1.0;

  for (const Group& gr : groups) {
    const int64_t rows = gr.rows, cols = gr.cols;
    const int64_t k = dion ? k_rows(hp->row_fraction, rows) : rows;
    const Geo g = make_geo(k, cols, sto);      // the matrix NS runs on: k x cols
    for (size_t c0 = 0; c0 < gr.idx.size(); c0 += kChunk) {
      const int c = (int)((gr.idx.size() - c0) < (size_t)kChunk ? gr.idx.size() - c0 : kChunk);
      PtrPack Wp = {}, Mp = {}, Gp = {}, Vp = {};
      for (int i = 0; i < c; ++i) {
        const mns_matrix& mm = mats[gr.idx[c0 + i]];
        Wp.p[i] = mm.W;
        Mp.p[i] = mm.M;
        Gp.p[i] = const_cast<void*>(mm.G);
        Vp.p[i] = mm.v;
      }
      st = step_chunk(g, c, rows, cols, k, hp, Wp, Mp, &Gp, nullptr, Vp, workspace, s);
      if (st != MNS_OK) return st;
    }
  }
  return MNS_OK;
}

// ---- standalone orthogonalisation ------------------------------------------------------------

static size_t ns_bytes(const Geo& g, int c, int kind, int64_t rows, int64_t cols,
                       NsBuffers* b, double** partials, float** xscale, void* base,
                       size_t gemm_cap = kGemmScratchBytes) {
  Carver cv(base);
  NsBuffers tmp;
  NsBuffers& nb = b ? *b : tmp;
  double* p = cv.take<double>((size_t)c * norm_blocks(rows * cols));
  float* x = cv.take<float>((size_t)c);
  carve_ns(cv, g, c, kind, nb, gemm_cap);
  if (partials) *partials = p;
  if (xscale) *xscale = x;
  return cv.off + 256;
}

mns_status mns_ns_workspace_size(int dtype, int64_t batch, int64_t rows, int64_t cols, int kind,
                                 size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  mns_status st = check_dtype(dtype);
  if (st != MNS_OK) return st;
  st = check_shape(batch, rows, cols);
  if (st != MNS_OK) return st;
  st = check_iterate(rows, cols, dtype == MNS_BF16 ? Store::BF16 : Store::F32);
  if (st != MNS_OK) return st;
  if (kind != MNS_NS_STANDARD && kind != MNS_NS_GRAM) return MNS_ERR_PARAM;
  const Geo g = make_geo(rows, cols, dtype == MNS_BF16 ? Store::BF16 : Store::F32);
  const int c = batch < kChunk ? (int)batch : kChunk;
  *bytes = ns_bytes(g, c, kind, rows, cols, nullptr, nullptr, nullptr, nullptr);
  return MNS_OK;
}

// Argument checks shared by the orthogonalisation entry points (everything but the workspace).
static mns_status check_orthogonalize(const void* X, void* O, int dtype, int64_t batch,
                                      int64_t rows, int64_t cols, int T, const float* abc,
                                      int kind, uint32_t restart_mask) {
  mns_status st = check_dtype(dtype);
  if (st != MNS_OK) return st;
  st = check_shape(batch, rows, cols);
  if (st != MNS_OK) return st;
  st = check_iterate(rows, cols, dtype == MNS_BF16 ? Store::BF16 : Store::F32);
  if (st != MNS_OK) return st;
  if (!X || !O) return MNS_ERR_NULL;
  st = check_ns(T, abc, kind, restart_mask);
  if (st != MNS_OK) return st;
  if (!aligned(X, 16) || !aligned(O, 16)) return MNS_ERR_PARAM;
  return MNS_OK;
}

// The orthogonalisation of `batch` matrices in chunks of at most `cmax`, each chunk's
// buffers carved from `ws` (split-k scratch capped at gemm_cap): per chunk the Frobenius
// norm, the normalised iterate, T iterations (standard or Gram), and the export to O.
static mns_status run_orthogonalize(const void* X, void* O, Store sto, const Geo& g,
                                    int64_t batch, int64_t rows, int64_t cols, int T,
                                    const float* abc, int kind, uint32_t restart_mask, void* ws,
                                    int cmax, size_t gemm_cap, hipStream_t s) {
  const size_t esz = sto == Store::BF16 ? 2 : 4;
  for (int64_t b0 = 0; b0 < batch; b0 += cmax) {
    const int c = (int)((batch - b0) < cmax ? batch - b0 : cmax);
    NsBuffers nb;
    double* partials = nullptr;
    float* xscale = nullptr;
    ns_bytes(g, c, kind, rows, cols, &nb, &partials, &xscale, ws, gemm_cap);
    const bool km = kmajor_ns(g, c, nb);
    const char* xin = static_cast<const char*>(X) + (size_t)b0 * rows * cols * esz;
    char* out = static_cast<char*>(O) + (size_t)b0 * rows * cols * esz;
    const double all = (double)c * rows * cols, ss = (double)esz, es = elem_bytes(g.elem);
    const int nblk = norm_blocks(rows * cols);
    MNS_HIP(timed("sumsq", 0, all * ss, s, [&] {
      return sumsq(xin, sto, c, rows * cols, partials, s); }));
    MNS_HIP(timed("finalize_scale", 0, 4.0 * c * nblk, s, [&] {
      return finalize_scale(partials, nblk, c, g.S, xscale, s); }));
    MNS_HIP(timed("normalize", 0, all * (ss + (km ? 1.0 : 2.0) * es), s, [&] {
      return normalize(nullptr, xin, false, sto, c, rows, cols, xscale, g.elem,
                       straight(g, nb, km), transposed(g, nb, km), g.rows_p, g.cols_p, s); }));
    void* res = nullptr;
    const mns_status st = run_ns(g, c, nb, kind, T, abc, restart_mask, s, &res);
    if (st != MNS_OK) return st;
    MNS_HIP(timed("export", 0, all * (ss + es), s, [&] {
      return export_output(res, g.elem, g.rows_p, g.cols_p, c, rows, cols, 1.0f / g.S, out,
                           sto, s); }));
  }
  return MNS_OK;
}

static mns_status orthogonalize(const void* X, void* O, int dtype, int64_t batch, int64_t rows,
                                int64_t cols, int T, const float* abc, int kind,
                                uint32_t restart_mask, void* ws, size_t ws_bytes, void* stream) {
  mns_status st = check_orthogonalize(X, O, dtype, batch, rows, cols, T, abc, kind, restart_mask);
  if (st != MNS_OK) return st;
  const Store sto = dtype == MNS_BF16 ? Store::BF16 : Store::F32;
  const Geo g = make_geo(rows, cols, sto);
  const int cmax = batch < kChunk ? (int)batch : kChunk;
  st = check_ws(ws, ws_bytes, ns_bytes(g, cmax, kind, rows, cols, nullptr, nullptr, nullptr, nullptr));
  if (st != MNS_OK) return st;
  return run_orthogonalize(X, O, sto, g, batch, rows, cols, T, abc, kind, restart_mask, ws, cmax,
                           kGemmScratchBytes, static_cast<hipStream_t>(stream));
}

// ---- allocation-free standard NS (for callers that cannot allocate) ---------------------
//
// The same computation as ns_orthogonalize, with every buffer carved from one file-scope
// device array instead of a caller workspace. Each GPU the library runs on holds its own
// copy until the process ends. Host code never uses the array's name as an address: the
// first call on a device looks up that device's copy with hipGetSymbolAddress (with the
// device current) and keeps the pointer.
constexpr size_t kNoAllocScratchBytes = size_t(64) << 20;
static __device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

static constexpr int kMaxDevices = 64;
static std::mutex g_scratch_mu;
static void* g_scratch_ptr[kMaxDevices] = {};

// This device's copy of `scratch` (looked up once per device). The stream, if given, must
// belong to the current device: the array's address is the current device's.
static mns_status scratch_on_current_device(hipStream_t stream, void** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MNS_ERR_HIP;
  if (stream) {
    int sdev = -1;
    if (hipStreamGetDevice(stream, &sdev) != hipSuccess) return MNS_ERR_HIP;
    if (sdev != dev) return MNS_ERR_PARAM;
  }
  std::lock_guard<std::mutex> lk(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return MNS_ERR_HIP;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return MNS_OK;
}

// Matrices per chunk and split-k scratch cap so that one chunk's buffers fit in `scratch`:
// the largest chunk (<= kChunk) whose buffers fit with the full split-k scratch of the
// workspace path; else one matrix per chunk with what space remains for split-k parts.
// False when one matrix's buffers alone do not fit.
static bool noalloc_plan(const Geo& g, int64_t batch, int64_t rows, int64_t cols, int* cmax,
                  size_t* gemm_cap) {
  const int hi = batch < kChunk ? (int)batch : kChunk;
  for (int c = hi; c >= 1; --c) {
    if (ns_bytes(g, c, MNS_NS_STANDARD, rows, cols, nullptr, nullptr, nullptr, nullptr) <=
        kNoAllocScratchBytes) {
      *cmax = c;
      *gemm_cap = kGemmScratchBytes;
      return true;
    }
  }
  const size_t base = ns_bytes(g, 1, MNS_NS_STANDARD, rows, cols, nullptr, nullptr, nullptr,
                               nullptr, 0);
  if (base > kNoAllocScratchBytes) return false;
  *cmax = 1;
  *gemm_cap = (kNoAllocScratchBytes - base) & ~size_t(255);
  return true;
}

mns_status ns_orthogonalize_noalloc(const void* X, void* O, int dtype, int64_t batch,
                                    int64_t rows, int64_t cols, int T, const float* abc,
                                    void* stream) {
  mns_status st = check_orthogonalize(X, O, dtype, batch, rows, cols, T, abc, MNS_NS_STANDARD, 0u);
  if (st != MNS_OK) return st;
  const Store sto = dtype == MNS_BF16 ? Store::BF16 : Store::F32;
  const Geo g = make_geo(rows, cols, sto);
  int cmax = 0;
  size_t gemm_cap = 0;
  if (!noalloc_plan(g, batch, rows, cols, &cmax, &gemm_cap)) return MNS_ERR_WORKSPACE;
  void* ws = nullptr;
  st = scratch_on_current_device(static_cast<hipStream_t>(stream), &ws);
  if (st != MNS_OK) return st;
  return run_orthogonalize(X, O, sto, g, batch, rows, cols, T, abc, MNS_NS_STANDARD, 0u, ws, cmax,
                           gemm_cap, static_cast<hipStream_t>(stream));
}

mns_status ns_orthogonalize(const void* X, void* O, int dtype, int64_t batch, int64_t rows,
                            int64_t cols, int T, const float* abc, void* workspace,
                            size_t workspace_bytes, void* stream) {
  return orthogonalize(X, O, dtype, batch, rows, cols, T, abc, MNS_NS_STANDARD, 0u, workspace,
                       workspace_bytes, stream);
}

mns_status gram_ns_orthogonalize(const void* X, void* O, int dtype, int64_t batch, int64_t rows,
                                 int64_t cols, int T, const float* abc, uint32_t restart_mask,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  return orthogonalize(X, O, dtype, batch, rows, cols, T, abc, MNS_NS_GRAM, restart_mask,
                       workspace, workspace_bytes, stream);
}

// ---- standalone NorMuon ------------------------------------------------------------------------

static size_t normuon_bytes(int64_t batch, int64_t rows, float** part, float** rowscale,
                            double** fin, void* base) {
  Carver cv(base);
  float* p = cv.take<float>((size_t)batch * rows);
  float* r = cv.take<float>((size_t)batch * rows);
  double* f = cv.take<double>((size_t)batch * 2 * normuon_blocks(rows));
  if (part) *part = p;
  if (rowscale) *rowscale = r;
  if (fin) *fin = f;
  return cv.off + 256;
}

mns_status mns_normuon_workspace_size(int64_t batch, int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  const mns_status st = check_shape(batch, rows, cols);
  if (st != MNS_OK) return st;
  *bytes = normuon_bytes(batch, rows, nullptr, nullptr, nullptr, nullptr);
  return MNS_OK;
}

mns_status normuon_scale(void* O, int dtype, int64_t batch, int64_t rows, int64_t cols, float* v,
                         float beta2, float eps, void* workspace, size_t workspace_bytes,
                         void* stream) {
  mns_status st = check_dtype(dtype);
  if (st != MNS_OK) return st;
  st = check_shape(batch, rows, cols);
  if (st != MNS_OK) return st;
  if (!O || !v) return MNS_ERR_NULL;
  if (!(beta2 >= 0.f && beta2 <= 1.f) || !(eps >= 0.f) || !std::isfinite(eps)) return MNS_ERR_PARAM;
  if (!aligned(O, 16) || !aligned(v, 4)) return MNS_ERR_PARAM;
  if (batch > 65535) return MNS_ERR_SHAPE;
  st = check_ws(workspace, workspace_bytes,
                normuon_bytes(batch, rows, nullptr, nullptr, nullptr, nullptr));
  if (st != MNS_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Store sto = dtype == MNS_BF16 ? Store::BF16 : Store::F32;
  float *part = nullptr, *rowscale = nullptr;
  double* fin = nullptr;
  normuon_bytes(batch, rows, &part, &rowscale, &fin, workspace);
  const double all = (double)batch * rows * cols, ss = sto == Store::BF16 ? 2.0 : 4.0;
  MNS_HIP(timed("row_sumsq_stored", 0, all * ss, s, [&] {
    return row_sumsq_stored(O, sto, (int)batch, rows, cols, part, s); }));
  MNS_HIP(timed("normuon_finalize", 0, 4.0 * batch * rows * 4, s, [&] {
    return normuon_finalize(part, 1, (int)batch, rows, cols, nullptr, v, rows, nullptr, beta2,
                            eps, 1.0f, 1.0f, rowscale, fin, s); }));
  MNS_HIP(timed("rowscale_apply", 0, 2.0 * all * ss, s, [&] {
    return rowscale_apply(O, sto, (int)batch, rows, cols, rowscale, s); }));
  return MNS_OK;
}

// ---- products grouped by expert ----------------------------------------------------------------

constexpr int64_t kMaxGroups = 65536;
constexpr int64_t kMaxRows = int64_t(1) << 30;      // row arithmetic in the kernels is 32-bit
constexpr int64_t kMaxPitch = int64_t(1) << 21;
constexpr int64_t kMaxTensorElems = int64_t(1) << 36;

static mns_status check_grouped(int dtype, int64_t groups, int64_t total_rows, int64_t n, int64_t k) {
  const mns_status st = check_dtype(dtype);
  if (st != MNS_OK) return st;
  if (groups < 1 || groups > kMaxGroups || total_rows < 0 || total_rows > kMaxRows)
    return MNS_ERR_SHAPE;
  return check_shape(1, n, k);
}

static Store store_of(int dtype) { return dtype == MNS_BF16 ? Store::BF16 : Store::F32; }

static size_t store_bytes(int dtype) { return dtype == MNS_BF16 ? 2 : 4; }

static mns_status run_grouped(GroupedDesc& d, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (grouped_blocks(d) > kMaxElems) return MNS_ERR_SHAPE;
  const size_t need = grouped_workspace(d);
  if (need) {
    const mns_status st = check_ws(workspace, workspace_bytes, need);
    if (st != MNS_OK) return st;
    d.workspace = static_cast<float*>(workspace);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  MNS_HIP(timed(grouped_name(d), 2.0 * d.total_rows * d.n * d.k, 0.0, s, [&] {
    return grouped(d, s); }));
  return MNS_OK;
}

mns_status mns_grouped_workspace_size(int weight_grad, int dtype, int64_t groups,
                                      int64_t total_rows, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  if (weight_grad != 0 && weight_grad != 1) return MNS_ERR_PARAM;
  const mns_status st = check_grouped(dtype, groups, total_rows, n, k);
  if (st != MNS_OK) return st;
  GroupedDesc d;
  d.store = store_of(dtype);
  d.groups = groups;
  d.total_rows = total_rows;
  d.n = n;
  d.k = k;
  d.weight_grad = weight_grad == 1;
  *bytes = grouped_workspace(d);
  if (!weight_grad) {                 // for either direction
    d.transpose_w = true;
    const size_t other = grouped_workspace(d);
    if (other > *bytes) *bytes = other;
  }
  return MNS_OK;
}

mns_status mns_grouped_layer_workspace_size(int input_grad, int dtype, int64_t groups,
                                            int64_t total_rows, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  if (input_grad != 0 && input_grad != 1) return MNS_ERR_PARAM;
  const mns_status st = check_grouped(dtype, groups, total_rows, n, k);
  if (st != MNS_OK) return st;
  *bytes = 0;
  if (total_rows == 0) return MNS_OK;
  GroupedDesc d;
  d.store = d.out_store = store_of(dtype);
  d.groups = groups;
  d.total_rows = total_rows;
  d.n = n;
  d.k = k;
  d.transpose_w = input_grad == 1;
  d.layer = true;
  for (int64_t pitch = 0; pitch < 2; ++pitch) {      // of operands on 16 bytes, and not
    d.lda = pitch;
    const size_t need = grouped_workspace(d);
    if (need > *bytes) *bytes = need;
  }
  return MNS_OK;
}

mns_status grouped_matmul(const void* X, int64_t ldx, const void* W, void* Y, int64_t ldy,
                          int dtype, const int64_t* offsets, int64_t groups, int64_t total_rows,
                          int64_t n, int64_t k, int transpose_w, int fill_rest, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const mns_status st = check_grouped(dtype, groups, total_rows, n, k);
  if (st != MNS_OK) return st;
  if (transpose_w != 0 && transpose_w != 1) return MNS_ERR_PARAM;
  if (fill_rest != 0 && fill_rest != 1) return MNS_ERR_PARAM;
  const int64_t in = transpose_w ? n : k, out = transpose_w ? k : n;
  if (ldx < in || ldx > kMaxPitch || ldy < out || ldy > kMaxPitch) return MNS_ERR_SHAPE;
  if (!W || !offsets || (total_rows > 0 && (!X || !Y))) return MNS_ERR_NULL;
  const size_t es = store_bytes(dtype);
  if (!aligned(X, es) || !aligned(W, es) || !aligned(Y, es) || !aligned(offsets, 8))
    return MNS_ERR_PARAM;
  if (total_rows == 0) return MNS_OK;
  GroupedDesc d;
  d.store = d.out_store = store_of(dtype);
  d.A = X; d.lda = ldx;
  d.B = W;
  d.C = Y; d.ldc = ldy;
  d.offsets = offsets;
  d.groups = groups;
  d.total_rows = total_rows;
  d.n = n;
  d.k = k;
  d.transpose_w = transpose_w == 1;
  d.fill_rest = fill_rest == 1;
  return run_grouped(d, workspace, workspace_bytes, stream);
}

mns_status grouped_weight_grad(const void* dY, int64_t lddy, const void* X, int64_t ldx,
                               int dtype, const int64_t* offsets, int64_t groups,
                               int64_t total_rows, int64_t n, int64_t k, const void* C, float beta,
                               void* G, int out_dtype, void* workspace, size_t workspace_bytes,
                               void* stream) {
  mns_status st = check_grouped(dtype, groups, total_rows, n, k);
  if (st != MNS_OK) return st;
  st = check_dtype(out_dtype);
  if (st != MNS_OK) return st;
  if (out_dtype != dtype && out_dtype != MNS_F32) return MNS_ERR_DTYPE;
  if (!std::isfinite(beta)) return MNS_ERR_PARAM;
  if (lddy < n || lddy > kMaxPitch || ldx < k || ldx > kMaxPitch) return MNS_ERR_SHAPE;
  if (!G || !offsets || (total_rows > 0 && (!dY || !X))) return MNS_ERR_NULL;
  const size_t es = store_bytes(dtype), os = store_bytes(out_dtype);
  if (!aligned(dY, es) || !aligned(X, es) || !aligned(G, os) || !aligned(C, os) ||
      !aligned(offsets, 8))
    return MNS_ERR_PARAM;
  GroupedDesc d;
  d.store = store_of(dtype);
  d.out_store = store_of(out_dtype);
  d.A = dY; d.lda = lddy;
  d.B = X; d.ldb = ldx;
  d.D = beta != 0.f ? C : nullptr;
  d.beta = beta;
  d.C = G;
  d.offsets = offsets;
  d.groups = groups;
  d.total_rows = total_rows;
  d.n = n;
  d.k = k;
  d.weight_grad = true;
  return run_grouped(d, workspace, workspace_bytes, stream);
}

// ---- layers of experts ---------------------------------------------------------------------------

static_assert((int)MNS_ACT_NONE == ACT_NONE && (int)MNS_ACT_RELU == ACT_RELU &&
              (int)MNS_ACT_RELU2 == ACT_RELU2 && (int)MNS_ACT_GELU == ACT_GELU &&
              (int)MNS_ACT_SILU == ACT_SILU, "one numbering");

static bool act_ok(int act) { return act >= MNS_ACT_NONE && act <= MNS_ACT_SILU; }

static bool pitch_ok(const void* p, int64_t ld, int64_t width) {
  return !p || (ld >= width && ld <= kMaxPitch);
}

// The byte range of rows x width elements, empty for no rows.
struct Range {
  uintptr_t lo, hi;
};
static Range range_of(const void* p, int64_t rows, int64_t ld, int64_t width, size_t es) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  if (!p || rows < 1) return {b, b};
  return {b, b + ((size_t)(rows - 1) * ld + width) * es};
}
static bool apart(const Range& a, const Range& b) { return a.hi <= b.lo || b.hi <= a.lo; }

mns_status grouped_linear(const void* X, int64_t ldx, const void* W, const void* bias, int activation,
                          const void* R, int64_t ldr, void* Z, int64_t ldz, void* Y, int64_t ldy,
                          int dtype, const int64_t* offsets, int64_t groups, int64_t total_rows,
                          int64_t n, int64_t k, int fill_rest, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const mns_status st = check_grouped(dtype, groups, total_rows, n, k);
  if (st != MNS_OK) return st;
  if (!act_ok(activation) || (fill_rest != 0 && fill_rest != 1)) return MNS_ERR_PARAM;
  if (ldx < k || ldx > kMaxPitch || ldy < n || ldy > kMaxPitch || !pitch_ok(R, ldr, n) ||
      !pitch_ok(Z, ldz, n))
    return MNS_ERR_SHAPE;
  if (Z && activation == MNS_ACT_NONE) return MNS_ERR_PARAM;
  if (!W || !offsets || (total_rows > 0 && (!X || !Y))) return MNS_ERR_NULL;
  const size_t es = store_bytes(dtype);
  if (!aligned(X, es) || !aligned(W, es) || !aligned(Y, es) || !aligned(bias, es) ||
      !aligned(R, es) || !aligned(Z, es) || !aligned(offsets, 8))
    return MNS_ERR_PARAM;
  const Range x = range_of(X, total_rows, ldx, k, es), w = range_of(W, groups * n, k, k, es),
              b = range_of(bias, groups, n, n, es), r = range_of(R, total_rows, ldr, n, es),
              z = range_of(Z, total_rows, ldz, n, es), y = range_of(Y, total_rows, ldy, n, es),
              o = range_of(offsets, groups + 1, 1, 1, 8);
  if (!apart(y, x) || !apart(y, w) || !apart(y, b) || !apart(y, z) || !apart(y, o) ||
      !apart(z, x) || !apart(z, w) || !apart(z, b) || !apart(z, r) || !apart(z, o) ||
      (!apart(y, r) && (Y != R || ldy != ldr)))
    return MNS_ERR_PARAM;
  if (total_rows == 0) return MNS_OK;
  GroupedDesc d;
  d.store = d.out_store = store_of(dtype);
  d.A = X; d.lda = ldx;
  d.B = W;
  d.C = Y; d.ldc = ldy;
  d.offsets = offsets;
  d.groups = groups;
  d.total_rows = total_rows;
  d.n = n;
  d.k = k;
  d.fill_rest = fill_rest == 1;
  d.layer = true;
  d.bias = bias;
  d.R = R; d.ldr = ldr;
  d.Z = Z; d.ldz = ldz;
  d.act = activation;
  return run_grouped(d, workspace, workspace_bytes, stream);
}

mns_status grouped_input_grad(const void* dY, int64_t lddy, const void* W, int activation,
                              const void* Z, int64_t ldz, const void* R, int64_t ldr, void* dX,
                              int64_t lddx, int dtype, const int64_t* offsets, int64_t groups,
                              int64_t total_rows, int64_t n, int64_t k, int fill_rest,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const mns_status st = check_grouped(dtype, groups, total_rows, n, k);
  if (st != MNS_OK) return st;
  if (!act_ok(activation) || (fill_rest != 0 && fill_rest != 1)) return MNS_ERR_PARAM;
  if (lddy < n || lddy > kMaxPitch || lddx < k || lddx > kMaxPitch || !pitch_ok(R, ldr, k) ||
      !pitch_ok(Z, ldz, k))
    return MNS_ERR_SHAPE;
  const bool act = activation != MNS_ACT_NONE;
  if (!act && Z) return MNS_ERR_PARAM;
  if (!W || !offsets || (total_rows > 0 && (!dY || !dX || (act && !Z)))) return MNS_ERR_NULL;
  const size_t es = store_bytes(dtype);
  if (!aligned(dY, es) || !aligned(W, es) || !aligned(dX, es) || !aligned(R, es) ||
      !aligned(Z, es) || !aligned(offsets, 8))
    return MNS_ERR_PARAM;
  const Range g = range_of(dY, total_rows, lddy, n, es), w = range_of(W, groups * n, k, k, es),
              r = range_of(R, total_rows, ldr, k, es), z = range_of(Z, total_rows, ldz, k, es),
              x = range_of(dX, total_rows, lddx, k, es), o = range_of(offsets, groups + 1, 1, 1, 8);
  if (!apart(x, g) || !apart(x, w) || !apart(x, o) || (!apart(x, r) && (dX != R || lddx != ldr)) ||
      (!apart(x, z) && (dX != Z || lddx != ldz)))
    return MNS_ERR_PARAM;
  if (total_rows == 0) return MNS_OK;
  GroupedDesc d;
  d.store = d.out_store = store_of(dtype);
  d.A = dY; d.lda = lddy;
  d.B = W;
  d.C = dX; d.ldc = lddx;
  d.offsets = offsets;
  d.groups = groups;
  d.total_rows = total_rows;
  d.n = n;
  d.k = k;
  d.transpose_w = true;
  d.fill_rest = fill_rest == 1;
  d.layer = true;
  d.R = R; d.ldr = ldr;
  d.Z = const_cast<void*>(Z); d.ldz = ldz;       // read only (transpose_w)
  d.act = activation;
  return run_grouped(d, workspace, workspace_bytes, stream);
}

static mns_status check_bias_grad(int64_t groups, int64_t total_rows, int64_t n) {
  if (groups < 1 || groups > kMaxGroups || total_rows < 0 || total_rows > kMaxRows || n < 1 ||
      n > kMaxDim || bias_grad_blocks(groups, total_rows, n) > kMaxElems)
    return MNS_ERR_SHAPE;
  return MNS_OK;
}

mns_status mns_grouped_bias_grad_workspace_size(int64_t groups, int64_t total_rows, int64_t n,
                                                size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  const mns_status st = check_bias_grad(groups, total_rows, n);
  if (st != MNS_OK) return st;
  *bytes = bias_grad_workspace(groups, total_rows, n);
  return MNS_OK;
}

mns_status grouped_bias_grad(const void* dY, int64_t lddy, int activation, const void* Z, int64_t ldz,
                             void* dZ, int64_t lddz, int dtype, const int64_t* offsets,
                             int64_t groups, int64_t total_rows, int64_t n, void* db, int out_dtype,
                             int fill_rest, void* workspace, size_t workspace_bytes, void* stream) {
  mns_status st = check_dtype(dtype);
  if (st != MNS_OK) return st;
  st = check_dtype(out_dtype);
  if (st != MNS_OK) return st;
  if (out_dtype != dtype && out_dtype != MNS_F32) return MNS_ERR_DTYPE;
  st = check_bias_grad(groups, total_rows, n);
  if (st != MNS_OK) return st;
  if (!act_ok(activation) || (fill_rest != 0 && fill_rest != 1)) return MNS_ERR_PARAM;
  if (lddy < n || lddy > kMaxPitch || !pitch_ok(Z, ldz, n) || !pitch_ok(dZ, lddz, n))
    return MNS_ERR_SHAPE;
  const bool act = activation != MNS_ACT_NONE;
  if (!act && Z) return MNS_ERR_PARAM;
  if (!db || !offsets || (total_rows > 0 && (!dY || (act && !Z)))) return MNS_ERR_NULL;
  const size_t es = store_bytes(dtype), os = store_bytes(out_dtype);
  if (!aligned(dY, es) || !aligned(Z, es) || !aligned(dZ, es) || !aligned(db, os) ||
      !aligned(offsets, 8))
    return MNS_ERR_PARAM;
  const Range g = range_of(dY, total_rows, lddy, n, es), z = range_of(Z, total_rows, ldz, n, es),
              x = range_of(dZ, total_rows, lddz, n, es), b = range_of(db, groups, n, n, os),
              o = range_of(offsets, groups + 1, 1, 1, 8);
  if (!apart(b, g) || !apart(b, z) || !apart(b, x) || !apart(b, o) || !apart(x, o) ||
      (!apart(x, g) && (dZ != dY || lddz != lddy)) || (!apart(x, z) && (dZ != Z || lddz != ldz)))
    return MNS_ERR_PARAM;
  BiasGradDesc d;
  d.store = store_of(dtype);
  d.out_store = store_of(out_dtype);
  d.dY = dY; d.lddy = lddy;
  d.Z = Z; d.ldz = ldz;
  d.dZ = dZ; d.lddz = lddz;
  d.db = db;
  d.offsets = offsets;
  d.groups = groups;
  d.total_rows = total_rows;
  d.n = n;
  d.act = activation;
  d.fill_rest = fill_rest == 1;
  const size_t need = bias_grad_workspace(groups, total_rows, n);
  if (need) {
    st = check_ws(workspace, workspace_bytes, need);
    if (st != MNS_OK) return st;
    d.workspace = static_cast<float*>(workspace);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double bytes = (double)total_rows * n * es * (1 + (Z ? 1 : 0) + (dZ ? 1 : 0));
  MNS_HIP(timed("grouped_bias_grad", 0, bytes, s, [&] { return bias_grad(d, s); }));
  return MNS_OK;
}

// ---- a router's bookkeeping ------------------------------------------------------------------------

static mns_status check_routed(int64_t assignments, int64_t experts) {
  return assignments >= 0 && assignments <= kMaxRows && experts >= 1 && experts <= kMaxRouted
             ? MNS_OK : MNS_ERR_SHAPE;
}

mns_status mns_expert_order_workspace_size(int64_t assignments, int64_t experts, size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  const mns_status st = check_routed(assignments, experts);
  if (st != MNS_OK) return st;
  *bytes = order_workspace(assignments, experts);
  return MNS_OK;
}

mns_status expert_order(const int64_t* ids, int64_t assignments, int64_t experts, int64_t* counts,
                        int64_t* offsets, int64_t* order, void* workspace, size_t workspace_bytes,
                        void* stream) {
  mns_status st = check_routed(assignments, experts);
  if (st != MNS_OK) return st;
  if (!counts || !offsets || (assignments > 0 && !ids)) return MNS_ERR_NULL;
  if (!aligned(ids, 8) || !aligned(counts, 8) || !aligned(offsets, 8) || !aligned(order, 8))
    return MNS_ERR_PARAM;
  const Range all[4] = {range_of(ids, assignments, 1, 1, 8), range_of(counts, experts, 1, 1, 8),
                        range_of(offsets, experts + 1, 1, 1, 8),
                        range_of(order, assignments, 1, 1, 8)};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (!apart(all[i], all[j])) return MNS_ERR_PARAM;
  const size_t need = order_workspace(assignments, experts);
  if (need) {
    st = check_ws(workspace, workspace_bytes, need);
    if (st != MNS_OK) return st;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  MNS_HIP(timed("expert_order", 0, 8.0 * assignments * (order ? 2 : 1), s, [&] {
    return mns::expert_order(ids, assignments, experts, counts, offsets, order, workspace, s); }));
  return MNS_OK;
}

mns_status mns_balance_workspace_size(int64_t tokens, int64_t experts, size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  const mns_status st = check_routed(tokens, experts);
  if (st != MNS_OK) return st;
  *bytes = balance_workspace(tokens, experts);
  return MNS_OK;
}

mns_status balance_loss(const void* logits, int64_t ldl, int dtype, const int64_t* ids, int64_t top,
                        const int64_t* counts, int64_t tokens, int64_t experts, float scale,
                        float* loss, void* dlogits, int64_t ldd, void* workspace,
                        size_t workspace_bytes, void* stream) {
  mns_status st = check_dtype(dtype);
  if (st != MNS_OK) return st;
  st = check_routed(tokens, experts);
  if (st != MNS_OK) return st;
  if (top < 1 || (tokens > 0 && top > kMaxRows / tokens)) return MNS_ERR_SHAPE;
  if (ldl < experts || ldl > kMaxPitch || !pitch_ok(dlogits, ldd, experts)) return MNS_ERR_SHAPE;
  if (!std::isfinite(scale)) return MNS_ERR_PARAM;
  if (!counts || !loss || (tokens > 0 && (!logits || !ids))) return MNS_ERR_NULL;
  const size_t es = store_bytes(dtype);
  if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(ids, 8) || !aligned(counts, 8) ||
      !aligned(loss, 4))
    return MNS_ERR_PARAM;
  const Range l = range_of(logits, tokens, ldl, experts, es),
              g = range_of(dlogits, tokens, ldd, experts, es),
              i = range_of(ids, tokens, top, top, 8), c = range_of(counts, experts, 1, 1, 8),
              o = range_of(loss, 1, 1, 1, 4);
  if (!apart(o, l) || !apart(o, g) || !apart(o, i) || !apart(o, c) || !apart(g, i) ||
      !apart(g, c) || (!apart(g, l) && (dlogits != logits || ldd != ldl)))
    return MNS_ERR_PARAM;
  const size_t need = balance_workspace(tokens, experts);
  if (need) {
    st = check_ws(workspace, workspace_bytes, need);
    if (st != MNS_OK) return st;
  }
  BalanceDesc d;
  d.store = store_of(dtype);
  d.logits = logits; d.ld = ldl;
  d.ids = ids;
  d.counts = counts;
  d.grad = dlogits; d.ldg = ldd;
  d.loss = loss;
  d.tokens = tokens;
  d.experts = experts;
  d.top = top;
  d.scale = scale;
  d.workspace = workspace;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double bytes = (double)tokens * (experts * es * (dlogits ? 2 : 1) + 8.0 * top);
  MNS_HIP(timed("balance_loss", 0, bytes, s, [&] { return balance(d, s); }));
  return MNS_OK;
}

// ---- global norm and clipping ----------------------------------------------------------------------

constexpr int kMaxTensors = 65536;

mns_status mns_clip_workspace_size(int count, size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  if (count < 1 || count > kMaxTensors) return MNS_ERR_SHAPE;
  *bytes = clip_workspace(count);
  return MNS_OK;
}

static mns_status run_clip(const mns_tensor* tensors, int count, bool scale, float max_norm, float eps,
                           float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (count < 1 || count > kMaxTensors) return MNS_ERR_SHAPE;
  if (!tensors || !norm) return MNS_ERR_NULL;
  if (scale && (!(max_norm >= 0.f) || !(eps >= 0.f) || !std::isfinite(eps))) return MNS_ERR_PARAM;
  if (!aligned(norm, 4)) return MNS_ERR_PARAM;
  double bytes = 0;
  std::vector<ClipTensor> list;
  std::vector<Range> outs;
  try {
    list.resize(count);
    outs.reserve(count + 1);               // and the norm
  } catch (...) {
    return MNS_ERR_PARAM;
  }
  for (int i = 0; i < count; ++i) {
    const mns_tensor& t = tensors[i];
    const mns_status st = check_dtype(t.dtype);
    if (st != MNS_OK) return st;
    if (t.numel < 0 || t.numel > kMaxTensorElems) return MNS_ERR_SHAPE;
    if (t.numel > 0 && (!t.in || (scale && !t.out))) return MNS_ERR_NULL;
    const size_t es = store_bytes(t.dtype);
    if (!aligned(t.in, es) || (scale && !aligned(t.out, es))) return MNS_ERR_PARAM;
    list[i] = {t.in, scale ? t.out : nullptr, t.numel, store_of(t.dtype)};
    bytes += (double)t.numel * es;
    if (scale && t.numel > 0) outs.push_back(range_of(t.out, 1, 1, t.numel, es));
  }
  if (scale) {
    const Range nr = range_of(norm, 1, 1, 1, 4);
    outs.push_back(nr);
    std::sort(outs.begin(), outs.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    for (size_t i = 1; i < outs.size(); ++i)
      if (outs[i - 1].hi > outs[i].lo) return MNS_ERR_PARAM;
    // An input may meet no output but its own, and that one only as a whole. The outputs lie apart, so
    // those that meet it are neighbours in the sorted list.
    for (int i = 0; i < count; ++i) {
      if (tensors[i].numel == 0) continue;
      const Range in = range_of(tensors[i].in, 1, 1, tensors[i].numel, store_bytes(tensors[i].dtype));
      auto it = std::lower_bound(outs.begin(), outs.end(), in.lo,
                                 [](const Range& r, uintptr_t v) { return r.hi <= v; });
      for (; it != outs.end() && it->lo < in.hi; ++it)
        if (tensors[i].in != tensors[i].out || it->lo != in.lo || it->hi != in.hi)
          return MNS_ERR_PARAM;
    }
  }
  const mns_status st = check_ws(workspace, workspace_bytes, clip_workspace(count));
  if (st != MNS_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  MNS_HIP(timed(scale ? "clip_grad_norm" : "grad_norm", 0, bytes * (scale ? 3 : 1), s, [&] {
    return clip_grads(list.data(), count, scale, max_norm, eps, norm,
                      static_cast<double*>(workspace), s); }));
  return MNS_OK;
}

mns_status grad_norm(const mns_tensor* tensors, int count, float* norm, void* workspace,
                     size_t workspace_bytes, void* stream) {
  return run_clip(tensors, count, false, 0.f, 0.f, norm, workspace, workspace_bytes, stream);
}

mns_status clip_grad_norm(const mns_tensor* tensors, int count, float max_norm, float eps, float* norm,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return run_clip(tensors, count, true, max_norm, eps, norm, workspace, workspace_bytes, stream);
}

// ---- gradient of the orthogonalisation ---------------------------------------------------------
//
// Per iteration (see ns_backward.hip for the formulas): A = X X^T (symmetric), K = E X^T,
// S = K + K^T, P = a I + b A + c A^2 (symmetric), K = A S, Q = b S + c (K + K^T), then
// E <- [P Q] [E; X] as one product of twice the depth, and X <- P X (not after the last
// iteration). E and X lie one above the other in V (and side by side in V^T), P and Q side by
// side in PQ, so no product needs its operands gathered.
//
// Short sides up to 256 run in float32 whatever the storage: rounding the iterate to float16 is
// the largest error, it grows along the smallest singular values, and small near-square matrices
// show it most (float16 against float64, rank 64 plus noise: 4.3e-3 at 64 and 256 square, 2.9e-3
// at 512; half a bfloat16 step is 3.9e-3). The float32 products there take a few microseconds.
constexpr int64_t kNsbF32Short = 256;
// Largest growth of a direction over the iterations that float16 can carry (2^14 of headroom
// above 1, 2^6 below the smallest value that matters).
constexpr double kNsbGrowthF16 = 1048576.0, kNsbGrowthF32 = 1e30;
// Largest sum of the terms of an update, P E + Q X, that its float32 sums can hold.
constexpr double kNsbTerms = 1e37;

static Geo nsb_geo(int64_t rows, int64_t cols, Store st) {
  Geo g = make_geo(rows, cols, st);
  if (g.n <= kNsbF32Short) {
    g.elem = Elem::F32;
    g.S = 1.0f;
  }
  return g;
}

struct NsbBuffers {
  void* V[2] = {};       // [E; X]: 2 n_p x m_p, pitch ld_x
  void* Vt[2] = {};      // [E^T X^T]: m_p x 2 n_p, pitch ld_t
  void* A = nullptr;     // n_p x n_p, pitch ld_q
  void* K = nullptr;
  void* Ssym = nullptr;
  void* PQ = nullptr;    // n_p x 2 n_p, pitch ld_t
  double* px = nullptr;
  double* pg = nullptr;
  double* scale = nullptr;
  double* dot = nullptr;
  float* gemm_scratch = nullptr;
  size_t gemm_scratch_bytes = 0;
  void* C2 = nullptr;    // few launches (nsb_fused): 2 n_p square, pitch ld_t; PQ too is then
  int64_t ld_t = 0, v_stride = 0, vt_stride = 0, q_stride = 0, pq_stride = 0;
};

// Small problems, bound by their launches: an iteration as three launches instead of eight (A, K and K^T;
// the n x n side; the update), for a third to a half more arithmetic. In us, eight launches against
// three, float32 (the first and last on the general product, padded to 256): 256x1024 402 / 235,
// 4 x 64x2048 589 / 517, 16 x 256x1024 861 / 953, 512x2048 639 / 535, 4 x 512x512 721 / 780. float16
// (kernels of its own that stop at n, so that a small n counts for more, and a third to a half of the
// error, k_nsb_square and k_nsb_update, for which a few per cent of time are given up at the limit):
// 333x1111 303 / 170, 16 of them 761 / 771, 8 x 300x3000 759 / 680, 512x8192 465 / 422, 4 x 512x2048
// 447 / 451, 8 x 512x1024 536 / 563, 3 x 512x4096 451 / 556 and more, 16 x 512x512 522 / 712 and more.
static bool nsb_fused(const Geo& g, int count) {
  if (g.n_p > 512) return false;
  if (g.elem != Elem::F16) return (double)count * g.n_p * g.n_p * (g.m_p + g.n_p) <= 8e8;
  const double n = (double)((g.n + 127) / 128 * 128);
  return count * n * n * n * (g.m + n) <= 1.7e12;
}

static size_t carve_nsb(void* base, const Geo& g, int count, NsbBuffers& b) {
  Carver cv(base);
  const size_t es = (size_t)elem_bytes(g.elem);
  const int nblk = norm_blocks(g.rows * g.cols);
  b.px = cv.take<double>((size_t)count * nblk);
  b.pg = cv.take<double>((size_t)count * nblk);
  b.scale = cv.take<double>((size_t)count * 4);
  b.dot = cv.take<double>((size_t)count * nsb_dot_blocks(g.rows));
  b.ld_t = padded_ld(2 * g.n_p);
  const bool own = g.elem == Elem::F16 && nsb_fused(g, count);    // nsb_update: [E; X; dX]
  b.v_stride = (own ? 3 : 2) * g.n_p * g.ld_x;
  b.vt_stride = g.m_p * b.ld_t;
  b.q_stride = g.n_p * g.ld_q;
  b.pq_stride = g.n_p * b.ld_t;
  for (int i = 0; i < 2; ++i) {
    b.V[i] = cv.take<char>(es * count * b.v_stride);
    b.Vt[i] = cv.take<char>(es * count * b.vt_stride);
  }
  if (nsb_fused(g, count)) {
    b.pq_stride *= own ? 3 : 2;
    b.C2 = cv.take<char>(es * count * b.pq_stride);
  } else {
    b.A = cv.take<char>(es * count * b.q_stride);
    b.K = cv.take<char>(es * count * b.q_stride);
    b.Ssym = cv.take<char>(es * count * b.q_stride);
  }
  b.PQ = cv.take<char>(es * count * b.pq_stride);
  // split-k parts: (output tiles) x (k-tiles / 8), capped as in carve_ns
  const size_t deep = (size_t)(g.m_p > 2 * g.n_p ? g.m_p : 2 * g.n_p) / 256;
  size_t scratch = (size_t)count * 4 * g.n_p * g.m_p * deep * sizeof(float);
  if (scratch > kGemmScratchBytes) scratch = kGemmScratchBytes;
  b.gemm_scratch = cv.take<float>(scratch / sizeof(float));
  b.gemm_scratch_bytes = scratch;
  return cv.off + 256;
}

static double pow2_floor(double x) { return std::ldexp(1.0, std::ilogb(x)); }

// Short sides up to 64 (kNsbSmall). Blocks per matrix: a block reads 32 KB of partial sums for each
// (about 0.3 us) and takes about 5 us for 64 columns, so sqrt(m / 4) of them balance the two; no more
// than two per CU over the whole chunk.
static NsbSmall nsb_small_plan(const Geo& g, int count) {
  NsbSmall d;
  d.n = g.n;
  d.m = g.m;
  d.ld = (g.m + 63) / 64 * 64;
  d.count = count;
  d.tall = g.tall;
  const int64_t tiles = d.ld / 64;
  int64_t blocks = std::llround(std::sqrt((double)g.m / 4.0));
  if (blocks * count > 512) blocks = 512 / count;
  if (blocks > tiles) blocks = tiles;
  if (blocks < 1) blocks = 1;
  const int64_t per = (tiles + blocks - 1) / blocks;
  d.cols_per = (int)(per * 64);
  d.blocks = (int)((tiles + per - 1) / per);
  return d;
}

static size_t carve_nsb_small(void* base, const Geo& g, int count, NsbBuffers& b, NsbSmall& d) {
  Carver cv(base);
  const int nblk = norm_blocks(g.rows * g.cols);
  d = nsb_small_plan(g, count);
  b.px = cv.take<double>((size_t)count * nblk);
  b.pg = cv.take<double>((size_t)count * nblk);
  b.scale = cv.take<double>((size_t)count * 4);
  b.dot = cv.take<double>((size_t)count * nsb_dot_blocks(g.rows));
  d.V = cv.take<float>((size_t)count * 2 * 64 * d.ld);
  for (float*& p : d.part) p = cv.take<float>((size_t)count * d.blocks * 2 * 64 * 64);
  if (g.tall) d.Et = cv.take<float>((size_t)count * g.m * 64);
  return cv.off + 256;
}

static size_t nsb_bytes(void* base, const Geo& g, int count, NsbBuffers& b, NsbSmall& d) {
  return g.n <= kNsbSmall ? carve_nsb_small(base, g, count, b, d) : carve_nsb(base, g, count, b);
}

// A call's: of its full chunks, or of the last one where that takes the form of nsb_fused and more.
static size_t nsb_need(const Geo& g, int64_t batch) {
  NsbBuffers b;
  NsbSmall d;
  if (batch <= kChunk) return nsb_bytes(nullptr, g, (int)batch, b, d);
  const size_t full = nsb_bytes(nullptr, g, kChunk, b, d);
  const int rest = (int)(batch % kChunk);
  const size_t last = rest ? nsb_bytes(nullptr, g, rest, b, d) : 0;
  return full > last ? full : last;
}

// Powers of two that scale the stored quantities of one iteration: E by e, X by S / u (u the power
// of two below the largest singular value it can have, 1 where that lies within a factor of 8 of 1),
// S and A S by kap, P by p, Q by q = p e / S (so that P E and Q X add up), with the bounds below 2^14.
// b and c are the coefficients for the iterate over u, b u^2 and c u^4; x is u over the next iteration's.
// gram (run_nsb_fused): of A, and of K on top of e / S, so that float16 holds A's small entries.
struct NsbScale {
  double e, kap, p, q, gram, b, c, x;
};

// Largest |x (a + b x^2 + c x^4)| for x in [0, s]: at s or where a + 3 b y + 5 c y^2 = 0, y = x^2.
static double poly_range(double s, double a, double b, double c) {
  double top = std::fabs(s * (a + s * s * (b + s * s * c)));
  const double disc = 9.0 * b * b - 20.0 * a * c;
  if (!(disc >= 0.0)) return top;
  const double w = -1.5 * b - std::copysign(0.5 * std::sqrt(disc), b);      // 5 c y = w or a = w y
  for (const double y : {w / (5.0 * c), a / w}) {
    if (!(y > 0.0 && y < s * s)) continue;                                  // (none where c or w is 0)
    const double v = std::fabs(std::sqrt(y) * (a + y * (b + y * c)));
    if (v > top) top = v;
  }
  return top;
}

// The scales of the T iterations and of the final direction, sc[T].e. A direction of norm 1 grows
// to at most L_t = max over s in [0, 1] of |f_t'(s)| and |f_t(s) / s| (the factors of the
// derivative of the composed polynomial f_t), and the singular values to sup |f_t|; f_t takes [0, 1] to
// all of [0, sup |f_t|] in magnitude, so the next sup is a single polynomial's. False when L or the
// terms of an update leave the range of the arithmetic.
static bool nsb_plan(int T, const float* abc, const Geo& g, NsbScale* sc) {
  const bool f16 = g.elem == Elem::F16;
  constexpr int kGrid = 2048;
  constexpr double kLeast = 0x1p-100;      // of L, 1 / p and of u over the one before: all may be gone
  double L = 1.0, sup = 1.0, u = 1.0;
  double f[kGrid], d[kGrid];
  for (int i = 0; i < kGrid; ++i) {
    f[i] = (i + 1.0) / kGrid;
    d[i] = 1.0;
  }
  double slope0 = 1.0;       // f_t'(0)
  for (int t = 0; t <= T; ++t) {
    const double lim = 16384.0;
    sc[t] = NsbScale{1.0, 1.0, 1.0, 1.0, 1.0, 0.0, 0.0, 1.0};
    if (!std::isfinite(L) || !std::isfinite(sup) || L > (f16 ? kNsbGrowthF16 : kNsbGrowthF32))
      return false;
    if (f16) sc[t].e = pow2_floor(lim / L);
    if (t == T) break;
    const double a = abc[3 * t], b0 = abc[3 * t + 1], c0 = abc[3 * t + 2];
    const double b = b0 * u * u, c = c0 * u * u * u * u, top = sup / u;
    sc[t].b = b;
    sc[t].c = c;
    const double s2 = top * top;
    const double pmax = std::fabs(a) + std::fabs(b) * s2 + std::fabs(c) * s2 * s2;
    const double qmax = (std::fabs(b) + 2.0 * std::fabs(c) * s2) * 2.0 * L * top;
    if (!(pmax * (L > 1.0 ? L : 1.0) + qmax * top < kNsbTerms)) return false;
    if (f16) {
      const double big = s2 > 1.0 ? s2 : 1.0;
      sc[t].kap = pow2_floor(lim / (2.0 * L * (top > 1.0 ? top : 1.0) * big));
      double p = 256.0;
      if (p * pmax > lim || (pmax > 0.0 && p * pmax < 1.0)) p = pow2_floor(lim / pmax);
      if (p > 1.0 / kLeast) p = 1.0 / kLeast;
      if (p * sc[t].e / g.S * qmax > lim) p = pow2_floor(lim * g.S / (sc[t].e * qmax));
      sc[t].p = p;
      sc[t].q = p * sc[t].e / g.S;
      // K <= e L top gram / S <= 2^14, A <= top S
      sc[t].gram = pow2_floor(g.S / (top > 1.0 ? top : 1.0));
    }
    slope0 *= a;
    L = std::fabs(slope0) > kLeast ? std::fabs(slope0) : kLeast;
    for (int i = 0; i < kGrid; ++i) {
      const double x = f[i], x2 = x * x;
      f[i] = x * (a + x2 * (b0 + x2 * c0));
      d[i] *= a + x2 * (3.0 * b0 + x2 * 5.0 * c0);
      const double s = (i + 1.0) / kGrid;
      if (std::fabs(d[i]) > L) L = std::fabs(d[i]);
      if (std::fabs(f[i]) / s > L) L = std::fabs(f[i]) / s;
      if (!std::isfinite(f[i]) || !std::isfinite(d[i])) return false;
    }
    sup = poly_range(sup, a, b0, c0);
    double next = 1.0;
    if (sup > 0.0 && !(sup > 0.125 && sup < 8.0)) next = pow2_floor(sup);
    if (next < u * kLeast) next = u * kLeast;
    if (t < T - 1) sc[t].x = u / next;
    u = next;
  }
  return true;
}

static mns_status nsb_check(int dtype, int64_t batch, int64_t rows, int64_t cols) {
  mns_status st = check_dtype(dtype);
  if (st != MNS_OK) return st;
  st = check_shape(batch, rows, cols);
  if (st != MNS_OK) return st;
  const Store sto = dtype == MNS_BF16 ? Store::BF16 : Store::F32;
  st = check_iterate(rows, cols, sto);
  if (st != MNS_OK) return st;
  // the products address [E; X] and [E^T X^T] with 32-bit byte offsets
  const Geo g = nsb_geo(rows, cols, sto);
  const int64_t v = 2 * g.n_p * g.ld_x, vt = g.m_p * padded_ld(2 * g.n_p);
  return (v > vt ? v : vt) * elem_bytes(g.elem) <= kMaxElems ? MNS_OK : MNS_ERR_SHAPE;
}

// Whether the products [P Q] [E; X] and P X read [E; X] as it is stored (gemm_kmajor_ok goes by the
// output's tiles, the same for both).
static bool nsb_kmajor(const Geo& g, int c, const NsbBuffers& b) {
  GemmDesc d;
  d.elem = g.elem;
  d.C = b.V[1];
  d.M = (int)g.n_p;
  d.N = (int)g.m_p;
  d.K = (int)g.n_p;
  d.batch = c;
  return gemm_kmajor_ok(d);
}

// The fused form of run_nsb for small problems (nsb_fused): [E; X] [E; X]^T, the n x n side, the
// update.
static mns_status run_nsb_fused(const Geo& g, int c, const NsbBuffers& b, int T, const float* abc,
                                const NsbScale* sc, hipStream_t s, void** out) {
  const int n = (int)g.n_p, m = (int)g.m_p;
  const double nn = (double)c * g.n * g.n;
  GemmDesc base;
  base.elem = g.elem;
  base.batch = c;
  base.partial = b.gemm_scratch;
  base.partial_bytes = b.gemm_scratch_bytes;
  // (more rows never turn a product away from its k-major operand)
  const bool km = nsb_kmajor(g, c, b), f16 = g.elem == Elem::F16;
  int cur = 0;
  for (int t = 0; t < T; ++t) {
    const bool last = t == T - 1;
    // C2 = [E; X] [E; X]^T gram / S^2: A times gram, K times gram e / S
    const float alpha = (float)sc[t].gram / (g.S * g.S);
    if (f16) {
      MNS_HIP(timed("nsb_gram", 3.0 * nn * g.m, 0.0, s, [&] {
        return nsb_gram(b.V[cur], g.ld_x, b.v_stride, b.C2, b.ld_t, b.pq_stride, c, (int)g.n, n,
                        g.m, alpha, s); }));
    } else {
      GemmDesc gram = base;
      gram.A = gram.B = b.V[cur];
      gram.lda = gram.ldb = g.ld_x;
      gram.sA = gram.sB = b.v_stride;
      gram.C = b.C2; gram.ldc = b.ld_t; gram.sC = b.pq_stride;
      gram.M = gram.N = 2 * n;
      gram.K = m;
      gram.sym = true;
      gram.alpha = alpha;
      MNS_HIP(timed_gemm(gram, 3.0 * nn * g.m, s));
    }
    // E' times sc[t + 1].e; Q X comes with e / S (of K) times S (of X): e, as P E does
    const float r = (float)(sc[t + 1].e / sc[t].e);
    const double gr = sc[t].gram;
    const double wide = r > sc[t].x ? r : sc[t].x;
    const double p = f16 ? sc[t].p / wide : 1.0;                           // a power of two
    MNS_HIP(timed("nsb_square", 3.0 * nn * g.n, 0.0, s, [&] {
      return nsb_square(b.C2, b.PQ, b.ld_t, b.pq_stride, g.elem, c, (int)g.n, n, abc[3 * t],
                        (float)(sc[t].b / gr), (float)(sc[t].c / (gr * gr)), r, (float)sc[t].x,
                        (float)p, t == 0 && f16 ? b.scale : nullptr, g.S, s); }));
    if (f16) {
      const bool flip = last && g.tall;
      MNS_HIP(timed("nsb_update", (last ? 4.0 : 6.0) * nn * g.m, 0.0, s, [&] {
        return nsb_update(b.PQ, b.ld_t, b.pq_stride, b.V[cur], g.ld_x, b.v_stride,
                          flip ? b.Vt[cur ^ 1] : b.V[cur ^ 1], flip ? b.ld_t : g.ld_x,
                          flip ? b.vt_stride : b.v_stride, c, (int)g.n, n, g.m, m, (float)(1.0 / p),
                          t == 0, last, flip, s); }));
      cur ^= 1;
      continue;
    }
    GemmDesc up = base;
    up.A = b.PQ; up.lda = b.ld_t; up.sA = b.pq_stride;
    if (km) {
      up.B = b.V[cur]; up.ldb = g.ld_x; up.sB = b.v_stride;
      up.b_kmajor = true;
    } else {
      up.B = b.Vt[cur]; up.ldb = b.ld_t; up.sB = b.vt_stride;
    }
    if (!last || !g.tall) {
      up.C = b.V[cur ^ 1]; up.ldc = g.ld_x; up.sC = b.v_stride;
    }
    if (last ? g.tall : !km) {
      up.Ct = b.Vt[cur ^ 1]; up.ldct = b.ld_t; up.sCt = b.vt_stride;
    }
    up.M = last ? n : 2 * n; up.N = m; up.K = 2 * n;
    MNS_HIP(timed_gemm(up, (last ? 4.0 : 6.0) * nn * g.m, s));
    cur ^= 1;
  }
  *out = g.tall ? b.Vt[cur] : b.V[cur];
  return MNS_OK;
}

// One chunk of `c` matrices on buffers b: the direction E_T is left in the stored layout.
static mns_status run_nsb(const Geo& g, int c, const NsbBuffers& b, int T, const float* abc,
                          const NsbScale* sc, hipStream_t s, void** out) {
  const size_t es = (size_t)elem_bytes(g.elem);
  const auto at = [&](void* p, int64_t elems) {
    return static_cast<void*>(static_cast<char*>(p) + (size_t)elems * es);
  };
  const int n = (int)g.n_p, m = (int)g.m_p;
  const int64_t xoff = g.n_p * g.ld_x;                   // X below E in V
  const double nn = (double)c * g.n * g.n;
  GemmDesc base;
  base.elem = g.elem;
  base.batch = c;
  base.partial = b.gemm_scratch;
  base.partial_bytes = b.gemm_scratch_bytes;
  const auto square = [&](const void* A, const void* B, int64_t ld, int64_t st, int K, void* C) {
    GemmDesc d = base;
    d.A = A; d.lda = ld; d.sA = st;
    d.B = B; d.ldb = ld; d.sB = st;
    d.C = C; d.ldc = g.ld_q; d.sC = b.q_stride;
    d.M = d.N = n;
    d.K = K;
    return d;
  };
  // [P Q] V[cur] (depth 2 n_p) or P X (depth n_p)
  const auto update = [&](bool direction, int cur, bool km, bool last) {
    GemmDesc d = base;
    d.A = b.PQ; d.lda = b.ld_t; d.sA = b.pq_stride;
    if (km) {
      d.B = direction ? b.V[cur] : at(b.V[cur], xoff);
      d.ldb = g.ld_x; d.sB = b.v_stride;
      d.b_kmajor = true;
    } else {
      d.B = direction ? b.Vt[cur] : at(b.Vt[cur], g.n_p);
      d.ldb = b.ld_t; d.sB = b.vt_stride;
    }
    const bool want_c = !last || !g.tall, want_t = last ? g.tall : !km;
    if (want_c) {
      d.C = direction ? b.V[cur ^ 1] : at(b.V[cur ^ 1], xoff);
      d.ldc = g.ld_x; d.sC = b.v_stride;
    }
    if (want_t) {
      d.Ct = direction ? b.Vt[cur ^ 1] : at(b.Vt[cur ^ 1], g.n_p);
      d.ldct = b.ld_t; d.sCt = b.vt_stride;
    }
    d.M = n; d.N = m; d.K = direction ? 2 * n : n;
    return d;
  };
  const bool km = nsb_kmajor(g, c, b);
  int cur = 0;
  for (int t = 0; t < T; ++t) {
    const bool last = t == T - 1;
    const double a = abc[3 * t], bb = sc[t].b, cc = sc[t].c;
    const void* E = b.V[cur];
    const void* X = at(b.V[cur], xoff);
    GemmDesc gram = square(X, X, g.ld_x, b.v_stride, m, b.A);
    gram.sym = true;
    gram.alpha = 1.0f / (g.S * g.S);
    MNS_HIP(timed_gemm(gram, nn * g.m, s));
    GemmDesc cross = square(E, X, g.ld_x, b.v_stride, m, b.K);
    cross.alpha = (float)(sc[t].kap / (sc[t].e * g.S));
    MNS_HIP(timed_gemm(cross, 2.0 * nn * g.m, s));
    MNS_HIP(timed("symmetrise", 0, nn * 2.0 * es, s, [&] {
      return symmetrise(b.K, g.ld_q, b.q_stride, nullptr, 0, 0, b.Ssym, g.ld_q, b.q_stride, g.elem,
                        c, g.n_p, 0.f, 1.f, s); }));
    GemmDesc poly = square(b.A, b.A, g.ld_q, b.q_stride, n, b.PQ);
    poly.ldc = b.ld_t; poly.sC = b.pq_stride;
    poly.sym = true;
    poly.alpha = (float)(sc[t].p * cc);
    poly.beta = (float)(sc[t].p * bb);
    poly.D = b.A; poly.ldd = g.ld_q; poly.sD = b.q_stride;
    poly.gamma = (float)(sc[t].p * a);
    poly.diag_limit = (int)g.n;
    MNS_HIP(timed_gemm(poly, nn * g.n, s));
    MNS_HIP(timed_gemm(square(b.A, b.Ssym, g.ld_q, b.q_stride, n, b.K), 2.0 * nn * g.n, s));
    const double qk = sc[t].q / sc[t].kap;
    MNS_HIP(timed("symmetrise", 0, nn * 3.0 * es, s, [&] {
      return symmetrise(b.K, g.ld_q, b.q_stride, b.Ssym, g.ld_q, b.q_stride, at(b.PQ, g.n_p),
                        b.ld_t, b.pq_stride, g.elem, c, g.n_p, (float)(qk * bb), (float)(qk * cc),
                        s); }));
    GemmDesc dir = update(true, cur, km, last);
    dir.alpha = (float)(sc[t + 1].e / (sc[t].p * sc[t].e));
    MNS_HIP(timed_gemm(dir, 4.0 * nn * g.m, s));
    if (!last) {
      GemmDesc upd = update(false, cur, km, false);
      upd.alpha = (float)(sc[t].x / sc[t].p);
      MNS_HIP(timed_gemm(upd, 2.0 * nn * g.m, s));
    }
    cur ^= 1;
  }
  *out = g.tall ? b.Vt[cur] : b.V[cur];
  return MNS_OK;
}

mns_status mns_ns_backward_workspace_size(int dtype, int64_t batch, int64_t rows, int64_t cols,
                                          size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  const mns_status st = nsb_check(dtype, batch, rows, cols);
  if (st != MNS_OK) return st;
  *bytes = nsb_need(nsb_geo(rows, cols, store_of(dtype)), batch);
  return MNS_OK;
}

mns_status ns_orthogonalize_backward(const void* X, const void* dO, void* dX, int dtype,
                                     int64_t batch, int64_t rows, int64_t cols, int T,
                                     const float* abc, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  mns_status st = nsb_check(dtype, batch, rows, cols);
  if (st != MNS_OK) return st;
  if (!X || !dO || !dX) return MNS_ERR_NULL;
  st = check_ns(T, abc, MNS_NS_STANDARD, 0u);
  if (st != MNS_OK) return st;
  if (!aligned(X, 16) || !aligned(dO, 16) || !aligned(dX, 16)) return MNS_ERR_PARAM;
  const Store sto = store_of(dtype);
  const Geo g = nsb_geo(rows, cols, sto);
  NsbScale sc[kMaxT + 1];
  if (!nsb_plan(T, abc, g, sc)) return MNS_ERR_PARAM;
  const int cmax = batch < kChunk ? (int)batch : kChunk;
  NsbBuffers b;
  NsbSmall small;
  st = check_ws(workspace, workspace_bytes, nsb_need(g, batch));
  if (st != MNS_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t esz = store_bytes(dtype);
  const int nblk = norm_blocks(rows * cols);
  for (int64_t b0 = 0; b0 < batch; b0 += cmax) {
    const int c = (int)((batch - b0) < cmax ? batch - b0 : cmax);
    const bool own = g.elem == Elem::F16 && nsb_fused(g, c);       // nsb_update, V alone
    nsb_bytes(workspace, g, c, b, small);
    const size_t off = (size_t)b0 * rows * cols * esz;
    const char* x = static_cast<const char*>(X) + off;
    const char* go = static_cast<const char*>(dO) + off;
    char* dx = static_cast<char*>(dX) + off;
    const double all = (double)c * rows * cols, ss = (double)esz, es = elem_bytes(g.elem);
    MNS_HIP(timed("sumsq", 0, all * ss, s, [&] {
      return sumsq(x, sto, c, rows * cols, b.px, s); }));
    MNS_HIP(timed("sumsq", 0, all * ss, s, [&] {
      return sumsq(go, sto, c, rows * cols, b.pg, s); }));
    MNS_HIP(timed("nsb_scales", 0, 16.0 * c * nblk, s, [&] {
      return nsb_scales(b.px, b.pg, nblk, c, g.S, sc[0].e, own, b.scale, s); }));
    if (g.n <= kNsbSmall) {
      MNS_HIP(timed("nsb_small_load", 0, all * 2.0 * (ss + es), s, [&] {
        return nsb_small_load(small, x, go, sto, b.scale, s); }));
      const double nn = (double)c * g.n * g.n;
      for (int t = 0; t < T; ++t)
        MNS_HIP(timed("nsb_small_step", nn * (9.0 * g.m + 3.0 * g.n), 0, s, [&] {
          return nsb_small_step(small, t, t == T - 1, abc[3 * t], (float)sc[t].b, (float)sc[t].c,
                                (float)sc[t].x, s); }));
      MNS_HIP(timed("nsb_finish", 0, all * (3.0 * ss + 2.0 * es), s, [&] {
        return nsb_finish(x, sto, g.tall ? small.Et : small.V, Elem::F32, c, rows, cols,
                          g.tall ? 64 : small.ld, g.tall ? g.m * 64 : 128 * small.ld, b.dot,
                          b.scale, 1.0, dx, s); }));
      continue;
    }
    const NsbDst v{b.V[0], g.ld_x, b.v_stride, g.n_p * g.ld_x};
    // [E^T X^T] only where the products read it
    const NsbDst vt{own || nsb_kmajor(g, c, b) ? nullptr : b.Vt[0], b.ld_t, b.vt_stride, g.n_p};
    MNS_HIP(timed("nsb_load", 0, all * 2.0 * (ss + 2.0 * es), s, [&] {
      return nsb_load(x, go, sto, c, rows, cols, b.scale, g.elem, g.rows_p, g.cols_p,
                      g.tall ? vt : v, g.tall ? v : vt, s); }));
    void* E = nullptr;
    st = nsb_fused(g, c) ? run_nsb_fused(g, c, b, T, abc, sc, s, &E)
                         : run_nsb(g, c, b, T, abc, sc, s, &E);
    if (st != MNS_OK) return st;
    MNS_HIP(timed("nsb_finish", 0, all * (3.0 * ss + 2.0 * es), s, [&] {
      return nsb_finish(x, sto, E, g.elem, c, rows, cols, g.tall ? b.ld_t : g.ld_x,
                        g.tall ? b.vt_stride : b.v_stride, b.dot, b.scale, 1.0 / sc[T].e, dx, s); }));
  }
  return MNS_OK;
}

// ---- the step of a stack of experts from their tokens ------------------------------------------

static mns_status check_step_grouped(int64_t groups, int64_t total_rows, int64_t rows,
                                     int64_t cols, const mns_hparams* hp) {
  if (!hp) return MNS_ERR_NULL;
  mns_status st = check_grouped(hp->dtype, groups, total_rows, rows, cols);
  if (st != MNS_OK) return st;
  mns_matrix one = {};
  one.rows = rows;
  one.cols = cols;
  st = validate_step(&one, 1, hp, false);
  if (st != MNS_OK) return st;
  return hp->row_fraction == 1.0 ? MNS_OK : MNS_ERR_PARAM;
}

static GroupedDesc step_grouped_desc(int64_t groups, int64_t total_rows, int64_t rows, int64_t cols,
                                     const mns_hparams* hp) {
  GroupedDesc d;
  d.store = store_of(hp->dtype);
  d.out_store = Store::F32;
  d.groups = groups;
  d.total_rows = total_rows;
  d.n = rows;
  d.k = cols;
  d.weight_grad = true;
  return d;
}

// The product's workspace is free again when the first chunk starts: one region serves both.
static size_t step_grouped_bytes(int64_t groups, int64_t total_rows, int64_t rows, int64_t cols,
                                 const mns_hparams* hp) {
  const size_t prod = grouped_workspace(step_grouped_desc(groups, total_rows, rows, cols, hp));
  StepWs w;
  const size_t step = carve_step(nullptr, make_geo(rows, cols, store_of(hp->dtype)),
                                 groups < kChunk ? (int)groups : kChunk, rows, cols, false, rows,
                                 hp->kind, w);
  return prod > step ? prod : step;
}

mns_status mns_grouped_step_workspace_size(int64_t groups, int64_t total_rows, int64_t rows,
                                           int64_t cols, const mns_hparams* hp, size_t* bytes) {
  if (!bytes) return MNS_ERR_NULL;
  const mns_status st = check_step_grouped(groups, total_rows, rows, cols, hp);
  if (st != MNS_OK) return st;
  *bytes = step_grouped_bytes(groups, total_rows, rows, cols, hp);
  return MNS_OK;
}

mns_status muon_step_grouped(void* W, float* M, float* v, const void* dY, int64_t lddy,
                             const void* X, int64_t ldx, const int64_t* offsets, int64_t groups,
                             int64_t total_rows, int64_t rows, int64_t cols, const mns_hparams* hp,
                             void* workspace, size_t workspace_bytes, void* stream) {
  mns_status st = check_step_grouped(groups, total_rows, rows, cols, hp);
  if (st != MNS_OK) return st;
  if (!W || !M || (hp->normuon && !v)) return MNS_ERR_NULL;
  if (!aligned(W, 16) || !aligned(M, 16) || !aligned(v, 4)) return MNS_ERR_PARAM;
  st = check_ws(workspace, workspace_bytes,
                step_grouped_bytes(groups, total_rows, rows, cols, hp));
  if (st != MNS_OK) return st;
  // M <- mu M + dY^T X (its checks of the tokens come before anything is enqueued)
  const GroupedDesc d = step_grouped_desc(groups, total_rows, rows, cols, hp);
  st = grouped_weight_grad(dY, lddy, X, ldx, hp->dtype, offsets, groups, total_rows, rows, cols, M,
                           hp->mu, M, MNS_F32, grouped_workspace(d) ? workspace : nullptr,
                           workspace_bytes, stream);
  if (st != MNS_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Geo g = make_geo(rows, cols, store_of(hp->dtype));
  const size_t ws = store_bytes(hp->dtype), elems = (size_t)rows * cols;
  for (int64_t e0 = 0; e0 < groups; e0 += kChunk) {
    const int c = (int)(groups - e0 < kChunk ? groups - e0 : kChunk);
    PtrPack Wp = {}, Mp = {}, Vp = {};
    for (int i = 0; i < c; ++i) {
      const size_t e = (size_t)(e0 + i);
      Wp.p[i] = static_cast<char*>(W) + e * elems * ws;
      Mp.p[i] = M + e * elems;
      Vp.p[i] = v ? v + e * rows : nullptr;
    }
    st = step_chunk(g, c, rows, cols, rows, hp, Wp, Mp, nullptr, M + (size_t)e0 * elems, Vp,
                    workspace, s);
    if (st != MNS_OK) return st;
  }
  return MNS_OK;
}

mns_status mns_profile_begin(void) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  for (ProfRec& r : g_prof) {
    (void)hipEventDestroy(r.a);
    (void)hipEventDestroy(r.b);
  }
  g_prof.clear();
  g_prof_failed = false;
  g_prof_on.store(true, std::memory_order_release);
  return MNS_OK;
}

mns_status mns_profile_set_flush(void* buffer, size_t bytes) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  if (!g_prof_on.load()) return MNS_ERR_PARAM;
  if (buffer && !aligned(buffer, 16)) return MNS_ERR_PARAM;
  g_flush_buf = bytes ? buffer : nullptr;
  g_flush_bytes = buffer ? bytes : 0;
  return MNS_OK;
}

mns_status mns_profile_end(mns_kernel_stat* out, int capacity, int* count) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  if (!g_prof_on.load()) return MNS_ERR_PARAM;
  g_prof_on.store(false, std::memory_order_release);
  g_flush_buf = nullptr;
  g_flush_bytes = 0;
  std::vector<mns_kernel_stat> stats;
  bool ok = !g_prof_failed;
  for (ProfRec& r : g_prof) {
    float ms = 0.f;
    if (hipEventSynchronize(r.b) != hipSuccess || hipEventElapsedTime(&ms, r.a, r.b) != hipSuccess)
      ok = false;
    (void)hipEventDestroy(r.a);
    (void)hipEventDestroy(r.b);
    mns_kernel_stat* st = nullptr;
    for (auto& x : stats)
      if (std::strncmp(x.name, r.name, sizeof(x.name)) == 0) st = &x;
    if (!st) {
      mns_kernel_stat z = {};
      std::strncpy(z.name, r.name, sizeof(z.name) - 1);
      try {
        stats.push_back(z);
      } catch (...) {
        ok = false;
        continue;
      }
      st = &stats.back();
    }
    st->launches += 1;
    st->ms += ms;
    st->flops += r.flops;
    st->bytes += r.bytes;
  }
  g_prof.clear();
  if (count) *count = (int)stats.size();
  for (int i = 0; i < (int)stats.size() && i < capacity && out; ++i) out[i] = stats[i];
  return ok ? MNS_OK : MNS_ERR_HIP;
}

}  // extern "C"
