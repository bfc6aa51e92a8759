// The gated delta rule of a Gated DeltaNet layer, outputs and state, gfx950
// ("Efficient LLM Challenge Results", hazards list: most of the target's layers
// are Gated DeltaNet; the update is the gated delta rule of the paper the pages
// cite, the one that gdn_state_commit applies to the accepted prefix):
//
//   S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
//       = alpha_t S_{t-1} + u_t k_t^T,   u_t = beta_t (v_t - alpha_t S_{t-1} k_t)
//   o_t = scale S_t q_t                  S [dv x dk], fp32
//
// Two forms:
//   recurrent  token by token with the state in registers (decode, the verify
//              block, fp32 inputs);
//   chunked    64 tokens at a time on the matrix cores (prompts).
//
// Recurrent.  A state row needs only itself, k_t and q_t, so a block takes 32
// rows of one head, 8 threads a row, every thread holding every 8th 16-byte
// chunk of its row (8 threads read one whole 128-byte line).  With
//   o_t = scale (alpha_t S_{t-1} q_t + u_t (k_t . q_t))
// both dot products of a step read S_{t-1} and their sums over the 8 threads
// run side by side.  Tokens are staged in LDS 16 at a time, the next 16 on
// their way meanwhile.  Bound by the state's bytes for few tokens, by the steps'
// latency for many.
//
// Chunked.  Inside a chunk, with R[t][i] = prod_{i<j<=t} alpha_j (i <= t, running
// products: exact for any gate, zero included), G_t = prod_{j<=t} alpha_j and S
// the state before it,
//   u_t + sum_{i<t} beta_t R[t][i] (k_t.k_i) u_i = beta_t (v_t - G_t S k_t)
//   o_t = scale G_t S q_t + sum_{i<=t} scale R[t][i] (q_t.k_i) u_i
//   S' = G_63 S + sum_i R[63][i] u_i k_i^T
// so with L[t][i] = beta_t R[t][i] (k_t.k_i) and T = (I + L)^-1 (unit lower
// triangular), U = T diag(beta) (V - G K S^T).  What does not need the state, T
// diag(beta) and scale R (q.k), is computed for all chunks at once by
// gdn_chunk_kernel; gdn_scan_kernel then walks the chunks of a head.
#include "w4v_device.h"
#include "w4v_launch.h"

#include <algorithm>

namespace w4v {

namespace {

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __fp16 h16x4 __attribute__((ext_vector_type(4)));
#define W4V_LDS __attribute__((address_space(3)))

struct Seq {
  int start, T;      // first row and rows
};
__device__ __forceinline__ Seq seq_of(const GdnArgs& a, int b) {
  const int lo = min(max(a.cu[b], 0), a.N), hi = min(max(a.cu[b + 1], lo), a.N);
  return Seq{lo, hi - lo};
}

// ------------------------------------------------------------------ recurrent
constexpr int kTPR = 8;                    // threads per state row
constexpr int kRows = 32;                  // state rows per block
constexpr int kThreads = kTPR * kRows;
constexpr int kStage = 16;                 // tokens staged at a time

// sum over the 8 lanes of a state row: two steps inside the quad, one across its mirror
__device__ __forceinline__ float sum8(float v) {
  const auto dpp = [](float x, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x),
                                                                 decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
  v += dpp(v, std::integral_constant<int, 0x4E>{});    // quad_perm [2,3,0,1]
  v += dpp(v, std::integral_constant<int, 0x141>{});   // row_half_mirror
  return v;
}

template <int D, typename X>
__global__ __launch_bounds__(kThreads) void gdn_recurrent_kernel(GdnArgs a) {
  constexpr int CPT = D / kTPR, NC = CPT / 4;
  constexpr int kPer = kStage * D / kThreads;          // staged q (and k) values per thread
  __shared__ __attribute__((aligned(16))) float sq[kStage][D], sk[kStage][D];
  __shared__ float sv[kStage][kRows], sa[kStage], sb[kStage], skq[kStage];

  const int tid = threadIdx.x, row = tid / kTPR, r = tid % kTPR;
  const int h = blockIdx.y, b = blockIdx.z, row0 = blockIdx.x * kRows;
  const int hk = h / (a.H / a.Hk);
  const Seq sq_ = seq_of(a, b);
  const X* q = static_cast<const X*>(a.q) + (int64_t)sq_.start * a.ldq + hk * D;
  const X* k = static_cast<const X*>(a.k) + (int64_t)sq_.start * a.ldk + hk * D;
  const X* v = static_cast<const X*>(a.v) + (int64_t)sq_.start * a.ldv + h * D + row0;
  const float* al = a.alpha + (int64_t)sq_.start * a.H + h;
  const float* be = a.beta + (int64_t)sq_.start * a.H + h;
  X* o = static_cast<X*>(a.o) + (int64_t)sq_.start * a.ldo + h * D + row0;

  const int64_t soff = (((int64_t)b * a.H + h) * D + row0 + row) * D + 4 * r;
  float s[CPT];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(a.state + soff + 4 * kTPR * j);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[4 * j + e] = x[e];
  }

  X rq[kPer], rk[kPer], rv[2];
  float ra = 0.f, rb = 0.f;
  const auto fetch = [&](int t0) {                     // the stage's values, zeros behind the end
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int e = tid + u * kThreads, t = t0 + e / D, c = e % D;
      rq[u] = t < sq_.T ? q[(int64_t)t * a.ldq + c] : X(0);
      rk[u] = t < sq_.T ? k[(int64_t)t * a.ldk + c] : X(0);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = tid + u * kThreads, t = t0 + e / kRows, c = e % kRows;
      rv[u] = t < sq_.T ? v[(int64_t)t * a.ldv + c] : X(0);
    }
    if (tid < kStage) {
      const int t = t0 + tid;
      ra = t < sq_.T ? al[(int64_t)t * a.H] : 0.f;
      rb = t < sq_.T ? be[(int64_t)t * a.H] : 0.f;
    }
  };
  fetch(0);
  for (int t0 = 0; t0 < sq_.T; t0 += kStage) {
    __syncthreads();                                   // the previous stage has been read
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int e = tid + u * kThreads;
      sq[e / D][e % D] = (float)rq[u];
      sk[e / D][e % D] = (float)rk[u];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = tid + u * kThreads;
      sv[e / kRows][e % kRows] = (float)rv[u];
    }
    if (tid < kStage) {
      sa[tid] = ra;
      sb[tid] = rb;
    }
    __syncthreads();
    if (t0 + kStage < sq_.T) fetch(t0 + kStage);
    const int n = min(kStage, sq_.T - t0);
    for (int t = 0; t < n; ++t) {
      float kv[CPT], qv[CPT];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(&sk[t][4 * (j * kTPR + r)]);
        const f32x4 y = *reinterpret_cast<const f32x4*>(&sq[t][4 * (j * kTPR + r)]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kv[4 * j + e] = x[e];
          qv[4 * j + e] = y[e];
        }
      }
      float u = 0.f, w = 0.f, kq = 0.f;
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        u = __builtin_fmaf(s[j], kv[j], u);
        w = __builtin_fmaf(s[j], qv[j], w);
        kq = __builtin_fmaf(kv[j], qv[j], kq);
      }
      u = sum8(u);
      w = sum8(w);
      kq = sum8(kq);
      const float at = sa[t];
      const float cf = sb[t] * (sv[t][row] - at * u);
#pragma unroll
      for (int j = 0; j < CPT; ++j) s[j] = __builtin_fmaf(at, s[j], cf * kv[j]);
      if (r == 0) o[(int64_t)(t0 + t) * a.ldo + row] = (X)(a.scale * __builtin_fmaf(at, w, cf * kq));
    }
  }
  if (a.state_out != nullptr) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      *reinterpret_cast<f32x4*>(a.state_out + soff + 4 * kTPR * j) =
          f32x4{s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]};
  }
}

// ------------------------------------------------------------------ chunked
constexpr int kC = kGdnChunk;              // 64 tokens
constexpr int kLd = kC + 1;                // fp32 rows of the 64 x 64 tiles in LDS

// Workspace of one (chunk, head): the fragments of T diag(beta) and of
// scale R (q.k), as pairs of fp16 (x = hi + lo, 22 bits), in the order in which
// the scan's lanes take them, then G and R[63][.].
constexpr int kFrags = 6;                  // (row tile, 32-token step) pairs of a lower triangle
constexpr uint32_t kFragBytes = 1024;      // 64 lanes x 16 bytes
constexpr uint32_t kOffA = kFrags * 2 * kFragBytes;
constexpr uint32_t kOffGate = 2 * kOffA;
constexpr uint32_t kSlotBytes = kOffGate + 2 * kC * sizeof(float);
__device__ __forceinline__ constexpr int frag_of(int tt, int s) { return tt < 2 ? tt : 2 * tt - 2 + s; }

// Row rho of token tile tt is token tau: lane (col, grp) of an accumulator then
// holds, over the tile pair 2 s, 2 s + 1, the tokens 32 s + 8 grp + 0 .. 7, which are
// the k values the lane gives to the next product as its B operand: accumulators
// turn into operands without leaving the lane.  Rows of the state's tiles map to
// dk in the same way.
__device__ __forceinline__ int tau(int tt, int rho) {
  return 32 * (tt >> 1) + 8 * (rho >> 2) + 4 * (tt & 1) + (rho & 3);
}

// LDS rows of D fp16: chunk (16 bytes) c of row r sits at c ^ swz(r).  The
// operand reads (16 rows tau(tt, .), chunks 4 s + grp) meet no bank twice, the
// transposing reads (4 rows of 4 half chunks a 16-lane group) each bank twice,
// the least for half chunks.
template <int D>
__device__ __forceinline__ int swz(int r) {
  constexpr int sigma = 0x78;              // sigma = 0, 2, 3, 1 for row blocks 0 .. 3, two bits each
  const int sg = (sigma >> (2 * ((r >> 3) & 3))) & 3;
  return D == 128 ? 4 * (r & 3) + sg : 4 * ((r >> 1) & 1) + sg;
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(W4V_LDS const void*)p;
}

// Eight fp32 values (two accumulators' lanes) as fp16 pairs x = hi + lo.  The
// values are fixed in registers first: a product or sum that the compiler
// rounded to fp16 once for hi and through fp32 for lo would give a lo that
// belongs to another hi where the two roundings differ.
struct Pair {
  f16x8 hi, lo;
};
__device__ __forceinline__ Pair split(const f32x4& x, const f32x4& y) {
  Pair p;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v = e < 4 ? x[e & 3] : y[e & 3];
    asm("" : "+v"(v));
    const _Float16 h = (_Float16)v;
    p.hi[e] = h;
    p.lo[e] = (_Float16)(v - (float)h);
  }
  return p;
}

// 64 rows of D fp16 from global (row stride ld) into an LDS tile; rows at or past n are zeros
template <int D, int NT>
__device__ __forceinline__ void stage_rows(_Float16* dst, const _Float16* src, int64_t ld, int n) {
  constexpr int CH = D / 8;
#pragma unroll
  for (int u = 0; u < kC * CH / NT; ++u) {
    const int e = threadIdx.x + u * NT, r = e / CH, c = e % CH;
    f16x8 x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (_Float16)0.f;
    if (r < n) x = *reinterpret_cast<const f16x8*>(src + (int64_t)r * ld + 8 * c);
    *reinterpret_cast<f16x8*>(dst + r * D + ((c ^ swz<D>(r)) * 8)) = x;
  }
}

// acc += A B for 16 x 16 fp32 blocks in LDS (row strides kLd), on the fp32 matrix instruction
__device__ __forceinline__ void mm16(const float* A, const float* B, f32x4& acc) {
  const int col = threadIdx.x & 15, grp = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(A[col * kLd + 4 * kk + grp],
                                               B[(4 * kk + grp) * kLd + col], acc, 0, 0, 0);
}
__device__ __forceinline__ void put16(float* C, const f32x4& v, float sign) {
  const int col = threadIdx.x & 15, grp = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) C[(4 * grp + r) * kLd + col] = sign * v[r];
}

template <int D>
__global__ __launch_bounds__(256) void gdn_chunk_kernel(GdnArgs a, char* __restrict__ ws) {
  constexpr int DS = D / 32;
  __shared__ __attribute__((aligned(16))) _Float16 s_k[kC * D], s_q[kC * D];
  __shared__ float s_r[kC * kLd];          // R, then scale R (q.k)
  __shared__ float s_l[kC * kLd];          // L
  __shared__ float s_t[kC * kLd];          // T
  __shared__ float s_m[4][16 * kLd];
  __shared__ float s_beta[kC];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, grp = lane >> 4;
  const int slot = blockIdx.x, h = blockIdx.y, hk = h / (a.H / a.Hk);

  // the sequence whose chunks' slots hold this one: sequence b's start at cu[b] / 64 + b
  int b = 0;
  for (int b0 = 1; b0 < a.B; b0 += 64) {
    const int x = b0 + lane;
    b += __popcll(__ballot(x < a.B && min(max(a.cu[x], 0), a.N) / kC + x <= slot));
  }
  b = __builtin_amdgcn_readfirstlane(b);
  const Seq sq = seq_of(a, b);
  const int c = slot - (sq.start / kC + b);
  const int n = min(kC, sq.T - c * kC);
  if (c < 0 || n <= 0) return;
  const int64_t row0 = sq.start + (int64_t)c * kC;
  char* out = ws + ((int64_t)slot * a.H + h) * kSlotBytes;

  stage_rows<D, 256>(s_k, static_cast<const _Float16*>(a.k) + row0 * a.ldk + hk * D, a.ldk, n);
  stage_rows<D, 256>(s_q, static_cast<const _Float16*>(a.q) + row0 * a.ldq + hk * D, a.ldq, n);
  if (wave == 0) {
    const float al = lane < n ? a.alpha[(row0 + lane) * a.H + h] : 1.f;
    s_beta[lane] = lane < n ? a.beta[(row0 + lane) * a.H + h] : 0.f;
    float r = 0.f, g = 1.f;
    float* gate = reinterpret_cast<float*>(out + kOffGate);
#pragma unroll
    for (int t = 0; t < kC; ++t) {
      const float at = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, al), t));
      r = t == lane ? 1.f : r * at;        // zero until the column's own token
      g *= t <= lane ? at : 1.f;
      s_r[t * kLd + lane] = r;
    }
    gate[lane] = g;
    gate[kC + lane] = r;
  }
  __syncthreads();

  // L and scale R (q.k): wave w takes the 16 rows 16 w .. of both
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) kk[i] = qk[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto rows = [&](const _Float16* t, int r, int s) {
    return *reinterpret_cast<const f16x8*>(t + r * D + (((4 * s + grp) ^ swz<D>(r)) * 8));
  };
#pragma unroll
  for (int s = 0; s < DS; ++s) {
    const f16x8 ak = rows(s_k, 16 * wave + col, s), aq = rows(s_q, 16 * wave + col, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i > wave) continue;              // above the diagonal
      const f16x8 bk = rows(s_k, 16 * i + col, s);
      kk[i] = mfma16x16x32(ak, bk, kk[i]);
      qk[i] = mfma16x16x32(aq, bk, qk[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * wave + 4 * grp + r, j = 16 * i + col;
      const float d = s_r[t * kLd + j];
      s_l[t * kLd + j] = j < t ? s_beta[t] * d * kk[i][r] : 0.f;
      s_r[t * kLd + j] = j <= t ? a.scale * d * qk[i][r] : 0.f;
      s_t[t * kLd + j] = 0.f;
    }
  __syncthreads();

  // T = (I + L)^-1: the diagonal blocks by forward substitution (lane j: column
  // j, a row after the other), then the blocks below, one diagonal at a time:
  // T[i][j] = -T[i][i] sum_{j<=k<i} L[i][k] T[k][j]
  const int o16 = 16 * wave;
  if (lane < 16) {
    float x[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      float y = t == lane ? 1.f : 0.f;
#pragma unroll
      for (int i = 0; i < t; ++i) y = __builtin_fmaf(-s_l[(o16 + t) * kLd + o16 + i], x[i], y);
      x[t] = y;
      s_t[(o16 + t) * kLd + o16 + lane] = y;
    }
  }
  __syncthreads();
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    const int i = wave + d, j = wave;      // block (i, j) of this diagonal
    f32x4 m{0.f, 0.f, 0.f, 0.f};
    if (i < 4) {
      for (int k = j; k < i; ++k)
        mm16(s_l + 16 * i * kLd + 16 * k, s_t + 16 * k * kLd + 16 * j, m);
      put16(s_m[wave], m, 1.f);
    }
    __syncthreads();
    if (i < 4) {
      m = f32x4{0.f, 0.f, 0.f, 0.f};
      mm16(s_t + 16 * i * kLd + 16 * i, s_m[wave], m);
      put16(s_t + 16 * i * kLd + 16 * j, m, -1.f);
    }
    __syncthreads();
  }

  // fragments: wave w writes those of token tile w
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > wave / 2) continue;
    const int t = tau(wave, col), i0 = 32 * s + 8 * grp;
    f32x4 x0, x1, y0, y1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x0[e] = s_t[t * kLd + i0 + e] * s_beta[i0 + e];
      x1[e] = s_t[t * kLd + i0 + 4 + e] * s_beta[i0 + 4 + e];
      y0[e] = s_r[t * kLd + i0 + e];
      y1[e] = s_r[t * kLd + i0 + 4 + e];
    }
    const Pair x = split(x0, x1), y = split(y0, y1);
    char* f = out + (wave < 2 ? wave : 2 * wave - 2 + s) * 2 * kFragBytes + lane * 16;
    *reinterpret_cast<f16x8*>(f) = x.hi;
    *reinterpret_cast<f16x8*>(f + kFragBytes) = x.lo;
    *reinterpret_cast<f16x8*>(f + kOffA) = y.hi;
    *reinterpret_cast<f16x8*>(f + kOffA + kFragBytes) = y.lo;
  }
}

// The scan: a block walks the chunks of one head for NV tiles of 16 state rows
// (dv).  Per tile, a state wave holds S^T [D x 16] in its accumulators and
// computes X = K S^T, E = V - G X, U = T diag(beta) E and S' = G_63 S + (R[63] U)^T K;
// an output wave computes o = scale G Q S^T + A U beside it.  Both waves of a tile
// read the state and U as operands: the state wave leaves them in LDS as the
// fragments it uses itself.  One more wave copies the next chunk's K, Q, V rows
// and fragments into the other half of a double buffer (LDS DMA), so that
// nothing waits for memory inside a chunk.  Two barriers a chunk:
//   1  the chunk's copies have landed, S is in LDS
//   2  U is in LDS (and the output wave is done with S)
template <int D, int NV>
struct Scan {
  static constexpr int DS = D / 32, MT = D / 16;
  static constexpr int kThreads = 64 * (2 * NV + 1);
  static constexpr uint32_t kRowsB = kC * D * 2;             // K or Q rows
  static constexpr uint32_t kQ = kRowsB, kF = 2 * kRowsB;    // offsets in a buffer
  static constexpr uint32_t kGate = kF + 2 * kOffA;
  static constexpr uint32_t kV = kGate + 1024;
  static constexpr uint32_t kBuf = kV + kC * NV * 32;
  static constexpr uint32_t kS = 2 * kBuf;                   // [NV][DS][hi, lo] fragments
  static constexpr uint32_t kU = kS + NV * DS * 2 * kFragBytes;
  static constexpr uint32_t kBytes = kU + NV * 4 * kFragBytes;
  static_assert(kBytes <= 160 * 1024, "the scan's buffers exceed a CU's LDS");
};

__device__ __forceinline__ u32x4s rows_rsrc(const void* base, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4s{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu)),
                (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)bytes), 0x00020000u};
}

template <int D, int NV>
__global__ __launch_bounds__(64 * (2 * NV + 1), 1) void gdn_scan_kernel(GdnArgs a,
                                                                        const char* __restrict__ ws) {
  using L = Scan<D, NV>;
  constexpr int DS = L::DS, MT = L::MT;
  __shared__ __attribute__((aligned(1024))) unsigned char s_buf[L::kBytes];
  const uint32_t lds = lds_addr(s_buf);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, grp = lane >> 4;
  const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.H / a.Hk);
  const Seq sq = seq_of(a, b);
  const int slot0 = sq.start / kC + b;
  const int chunks = (sq.T + kC - 1) / kC;
  const int dv0 = blockIdx.x * NV * 16;

  const auto at = [&](uint32_t off) { return *(W4V_LDS f16x8*)(lds + off); };
  const auto frag = [&](uint32_t base, int i) { return at(base + i * kFragBytes + lane * 16); };
  // operand rows tau(tt, .) of K or Q, 32 dk of step s
  const auto rows = [&](uint32_t base, int tt, int s) {
    const int r = tau(tt, col);
    return at(base + r * D * 2 + ((4 * s + grp) ^ swz<D>(r)) * 16);
  };

  if (wave == 2 * NV) {
    // ---- the copying wave
    constexpr int CH = D / 8, CV = 2 * NV;
    const auto copy = [&](int c) {
      const uint32_t dst = lds + (c & 1) * L::kBuf;
      const int n = min(kC, sq.T - c * kC);
      const int64_t row0 = sq.start + (int64_t)c * kC;
      const auto* k = static_cast<const _Float16*>(a.k) + row0 * a.ldk + hk * D;
      const auto* q = static_cast<const _Float16*>(a.q) + row0 * a.ldq + hk * D;
      const auto* v = static_cast<const _Float16*>(a.v) + row0 * a.ldv + h * D + dv0;
      // rows at or past n lie behind the resource's end and become zeros
      const u32x4s rk = rows_rsrc(k, ((int64_t)(n - 1) * a.ldk + D) * 2);
      const u32x4s rq = rows_rsrc(q, ((int64_t)(n - 1) * a.ldq + D) * 2);
      const u32x4s rv = rows_rsrc(v, ((int64_t)(n - 1) * a.ldv + NV * 16) * 2);
      const u32x4s rf = rows_rsrc(ws + ((int64_t)(slot0 + c) * a.H + h) * kSlotBytes, kSlotBytes);
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        const int e = u * 64 + lane, r = e / CH, ch = (e % CH) ^ swz<D>(r);
        dma16(dst + u * 1024, rk, (uint32_t)(r * (int)a.ldk * 2 + ch * 16));
      }
#pragma unroll
      for (int u = 0; u < kOffA / 1024; ++u) dma16(dst + L::kF + u * 1024, rf, u * 1024 + lane * 16);
      dma16(dst + L::kGate, rf, kOffGate + lane * 16);
#pragma unroll
      for (int u = 0; u < CV; ++u) {
        const int e = u * 64 + lane;
        dma16(dst + L::kV + u * 1024, rv, (uint32_t)(e / CV * (int)a.ldv * 2 + e % CV * 16));
      }
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        const int e = u * 64 + lane, r = e / CH, ch = (e % CH) ^ swz<D>(r);
        dma16(dst + L::kQ + u * 1024, rq, (uint32_t)(r * (int)a.ldq * 2 + ch * 16));
      }
#pragma unroll
      for (int u = 0; u < kOffA / 1024; ++u)
        dma16(dst + L::kF + kOffA + u * 1024, rf, kOffA + u * 1024 + lane * 16);
    };
    if (chunks > 0) copy(0);
    for (int c = 0; c < chunks; ++c) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      lds_barrier();
      if (c + 1 < chunks) copy(c + 1);
      lds_barrier();
    }
  } else if (wave < NV) {
    // ---- a state wave: lane (dv, grp) holds dk 32 s + 8 grp + 0 .. 7 in tiles 2 s, 2 s + 1
    const int64_t soff = (((int64_t)b * a.H + h) * D + dv0 + wave * 16 + col) * D + 8 * grp;
    f32x4 st[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      st[m] = *reinterpret_cast<const f32x4*>(a.state + soff + 32 * (m >> 1) + 4 * (m & 1));
    Pair sp[DS];
    const auto publish = [&]() {
#pragma unroll
      for (int s = 0; s < DS; ++s) {
        sp[s] = split(st[2 * s], st[2 * s + 1]);
        const uint32_t f = lds + L::kS + (wave * DS + s) * 2 * kFragBytes + lane * 16;
        *(W4V_LDS f16x8*)f = sp[s].hi;
        *(W4V_LDS f16x8*)(f + kFragBytes) = sp[s].lo;
      }
    };
    publish();
    for (int c = 0; c < chunks; ++c) {
      const uint32_t buf = (c & 1) * L::kBuf;
      lds_barrier();
      f32x4 e[4], u[4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) e[tt] = u[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < DS; ++s)
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const f16x8 kf = rows(buf, tt, s);
          e[tt] = mfma16x16x32(kf, sp[s].hi, e[tt]);
          u[tt] = mfma16x16x32(kf, sp[s].lo, u[tt]);
        }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int t0 = 32 * (tt >> 1) + 8 * grp + 4 * (tt & 1);
        const f32x4 g = *(W4V_LDS f32x4*)(lds + buf + L::kGate + t0 * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v = (float)*(W4V_LDS _Float16*)(lds + buf + L::kV +
                                                      ((t0 + r) * NV * 16 + wave * 16 + col) * 2);
          e[tt][r] = v - g[r] * (e[tt][r] + u[tt][r]);
          u[tt][r] = 0.f;
        }
      }
      const Pair ep[2] = {split(e[0], e[1]), split(e[2], e[3])};
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int x = 0; x < 3; ++x)
#pragma unroll
          for (int tt = 2 * s; tt < 4; ++tt) {
            const f16x8 t = frag(buf + L::kF, frag_of(tt, s) * 2 + (x == 1));
            u[tt] = mfma16x16x32(t, x == 2 ? ep[s].lo : ep[s].hi, u[tt]);
          }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const Pair p = split(u[2 * s], u[2 * s + 1]);
        const uint32_t f = lds + L::kU + (wave * 2 + s) * 2 * kFragBytes + lane * 16;
        *(W4V_LDS f16x8*)f = p.hi;
        *(W4V_LDS f16x8*)(f + kFragBytes) = p.lo;
      }
      lds_barrier();
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int t0 = 32 * (tt >> 1) + 8 * grp + 4 * (tt & 1);
        const f32x4 d = *(W4V_LDS f32x4*)(lds + buf + L::kGate + (kC + t0) * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) u[tt][r] *= d[r];
      }
      const Pair up[2] = {split(u[0], u[1]), split(u[2], u[3])};
      const float gc = *(W4V_LDS float*)(lds + buf + L::kGate + (kC - 1) * 4);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[m][r] *= gc;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          // rows rho of tile m are dk 32 (m / 2) + 8 (rho / 4) + 4 (m & 1) + rho % 4
          f16x8 kt;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int t = 32 * s + 8 * grp + 4 * hf + (col >> 2);
            const int ch = 4 * (m >> 1) + (col & 3);
            const h16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4f16(
                (W4V_LDS h16x4*)(lds + buf + t * D * 2 + ((ch ^ swz<D>(t)) * 16) + 8 * (m & 1)));
#pragma unroll
            for (int i = 0; i < 4; ++i) kt[4 * hf + i] = (_Float16)x[i];
          }
          st[m] = mfma16x16x32(kt, up[s].hi, st[m]);
          st[m] = mfma16x16x32(kt, up[s].lo, st[m]);
        }
      if (c + 1 < chunks) publish();
    }
    if (a.state_out != nullptr) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
        *reinterpret_cast<f32x4*>(a.state_out + soff + 32 * (m >> 1) + 4 * (m & 1)) = st[m];
    }
  } else {
    // ---- an output wave
    const int tile = wave - NV;
    _Float16* out = static_cast<_Float16*>(a.o) + (int64_t)sq.start * a.ldo + h * D + dv0 + tile * 16 + col;
    for (int c = 0; c < chunks; ++c) {
      const uint32_t buf = (c & 1) * L::kBuf;
      const int n = min(kC, sq.T - c * kC);
      lds_barrier();
      f32x4 o[4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) o[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < DS; ++s) {
        const f16x8 sh = frag(L::kS, (tile * DS + s) * 2), sl = frag(L::kS, (tile * DS + s) * 2 + 1);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const f16x8 qf = rows(buf + L::kQ, tt, s);
          o[tt] = mfma16x16x32(qf, sh, o[tt]);
          o[tt] = mfma16x16x32(qf, sl, o[tt]);
        }
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int t0 = 32 * (tt >> 1) + 8 * grp + 4 * (tt & 1);
        const f32x4 g = *(W4V_LDS f32x4*)(lds + buf + L::kGate + t0 * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[tt][r] *= a.scale * g[r];
      }
      lds_barrier();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const f16x8 uh = frag(L::kU, (tile * 2 + s) * 2), ul = frag(L::kU, (tile * 2 + s) * 2 + 1);
#pragma unroll
        for (int x = 0; x < 3; ++x)
#pragma unroll
          for (int tt = 2 * s; tt < 4; ++tt) {
            const f16x8 t = frag(buf + L::kF + kOffA, frag_of(tt, s) * 2 + (x == 1));
            o[tt] = mfma16x16x32(t, x == 2 ? ul : uh, o[tt]);
          }
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int t0 = 32 * (tt >> 1) + 8 * grp + 4 * (tt & 1);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (t0 + r < n) out[((int64_t)c * kC + t0 + r) * a.ldo] = (_Float16)o[tt][r];
      }
    }
  }
}

}  // namespace

size_t gdn_forward_workspace(const GdnPlan& p, int N, int B, int H) {
  return p.chunked ? ((size_t)(N / kC) + B) * H * kSlotBytes : 0;
}

GdnPlan plan_gdn(int N, int max_t, int f32) { return GdnPlan{N > 0 && !f32 && max_t > 64}; }

template <int D>
static void launch_gdn(const GdnArgs& a, const GdnPlan& p, void* ws, hipStream_t stream) {
  if (p.chunked) {
    hipLaunchKernelGGL(gdn_chunk_kernel<D>, dim3(a.N / kC + a.B, a.H), dim3(256), 0, stream, a,
                       static_cast<char*>(ws));
    hipLaunchKernelGGL((gdn_scan_kernel<D, 2>), dim3(D / 32, a.H, a.B), dim3(Scan<D, 2>::kThreads), 0,
                       stream, a, static_cast<const char*>(ws));
  } else if (a.f32) {
    hipLaunchKernelGGL((gdn_recurrent_kernel<D, float>), dim3(D / kRows, a.H, a.B), dim3(kThreads), 0,
                       stream, a);
  } else {
    hipLaunchKernelGGL((gdn_recurrent_kernel<D, _Float16>), dim3(D / kRows, a.H, a.B),
                       dim3(kThreads), 0, stream, a);
  }
}

hipError_t launch_gdn_forward(const GdnArgs& a, const GdnPlan& p, void* ws, hipStream_t stream) {
  if (a.D == 128) launch_gdn<128>(a, p, ws, stream);
  else launch_gdn<64>(a, p, ws, stream);
  return hipGetLastError();
}

}  // namespace w4v
