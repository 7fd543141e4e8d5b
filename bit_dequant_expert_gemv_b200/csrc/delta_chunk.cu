// delta_chunk.cu — the gated delta rule over whole sequences, 64 tokens (a chunk) at a time, on the tensor cores.
//
// With G the running sum of g inside a chunk and S the state before it, the chunk's updates u solve a
// triangular system, and everything else is a matrix product:
//   L_ij = beta_i e^(G_i - G_j) k_i.k_j  (j < i),   T = (I + L)^-1
//   U = T [ beta (V - e^G (K S)) ],   out = scale [ e^G (Q S) + M U ],  M_ij = e^(G_i - G_j) q_i.k_j  (j <= i)
//   S <- e^(G_C) S + (e^(G_C - G) K)^T U
//
// One CTA carries one head of one sequence. Every product of the chain is taken transposed, with the state's
// columns as its 128 rows: a thread owns one of them and, between two products, reads its row from tensor
// memory, scales it, and writes it back as the next product's left operand. No value moves between threads on
// the way; the right operands (K and Q stacked, T, M, and K again, read across) are shared memory.
//   warps 0-3   the chain  S -> [K S | Q S] -> right-hand side -> U -> S, three products one after another
//   warps 4-11  one chunk ahead: norms, running decays, [K; Q] K^T, L, M and the inverse (blocks of 8, 16, 32,
//               64, binary32), into the other of two stages
//   warps 12-15 the outputs, from Q S and M U
// S stays in tensor memory in binary32. A chunk's increment is a product of its own and is added by the
// threads: sums over many chunks inside the tensor core would lose the rounding to nearest.
// Loops over blocks of 32 columns keep the code small: unrolled, it outgrew the instruction caches and every
// phase waited for its instructions (8 prompts, 8192 tokens, 64 heads: 614 us unrolled, 483 us in loops).
//
// Measured, 64 heads of 128 x 128: 8 packed prompts of 8192 tokens in all 450 to 575 us by their lengths, and by their
// order, in which the blocks start (the same eight lengths falling 414 us, mixed 454, rising 521: the longest runs alone
// at the end); one of 16384 tokens, binary16, 1725 us, one of 333 tokens 48 us. Latency bounds it, not a rate: a chunk
// is 6.7 us of products and of trips between tensor memory and registers that wait for one another, about as much in
// the chain as in the preparing warps, and one sequence has no more than a CTA a head, 64 for 148 SMs.
//
// Precision. Operands are binary16 with a power of two taken out of every row: keys and queries (16-bit
// inputs) are exact to 2^-25 of a row's largest value; binary32 operands (S, the right-hand side, U, T) are
// split into two binary16 parts, 22 bits, and products of two small parts are left out; norms, decays and
// gates multiply the binary32 results. For a bfloat16 output M, and U where it meets M, are rounded to binary16 (2^-12,
// its own rounding is 2^-8): they reach nothing but the output. A binary16 output (2^-11) has both parts of M and of
// U (with M in one its error was 1.4 times the rounding's), and the low parts of S where it meets Q.
//
// What is not finite. A product's zeros do not keep a NaN of a later token from the tokens before it, so nothing that is
// not finite goes into a product of tokens: such a key, query, gate or step size is taken as zeros and its place kept;
// a right-hand side from its column's first one on too (found by the maximum that is taken anyway). Results from
// there on, a query's own one, and the column's state are then made NaN.
#include "api.h"
#include "mixer.h"
#include "mma.cuh"
#include "tc05.cuh"

namespace fmoe {
namespace {

constexpr int C = 64;      // tokens of a chunk
constexpr int kChain = 128, kAux = 256, kOutputs = 128, kThreads = kChain + kAux + kOutputs;
constexpr int LD = C + 4;  // row stride of the binary32 matrices in shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTop = 14;   // a row's largest value is brought to [2^14, 2^15): 22 bits down to 2^-17 of it
enum { kBarFull = 1, kBarFree = 3, kBarAux = 5, kBarScales = 6, kBarTaken = 7, kBarOut = 8, kBarMain = 9, kBarRows = 10 };

// Tensor memory, columns: the state; its parts, then in their place its increment; K S, then the right-hand side,
// its parts, and U's parts for M; Q S, then M U; U, then its parts for the state; [K; Q] K^T. Parts take the
// place of the 32 values that they come from: 16 columns high, 16 low.
enum { kColS = 0, kColA = 128, kColP = 256, kColO = 320, kColU = 384, kColL = 448 };

template <int DK>
struct Smem {
  static constexpr int kPanels = DK / 64, kPanel = 128 * 128;  // [K; Q]: 128 rows of 64 columns each
  // a stage: operands; values; for each token e^G a, e^(G_C - G) a and the query's factor; a Scalars
  static constexpr int kKQ = 0, kTh = kKQ + kPanels * kPanel, kTl = kTh + C * 128, kM = kTl + C * 128, kMl = kM + C * 128;
  static constexpr int kV = kMl + C * 128, kCa = kV + C * 256, kW = kCa + C * 4, kOut = kW + C * 4, kEnd = kOut + C * 4;
  static constexpr int kStage = (kEnd + 32 + 1023) / 1024 * 1024;
  // behind two stages: rows as they come (32 bytes apart, for the banks), L and in its place the inverse, a product; running
  // decays with the keys' factors, gates, queries' factors, largest norms and entries, keys' factors with their decay to the end of their 16 tokens, row scales, first tokens of a row that are not finite
  static constexpr int kRow = DK * 2 + 32, kRaw = 2 * kStage, kL = kRaw + 2 * C * kRow;
  static constexpr int kY = kL + C * LD * 4, kG = kY + 32 * 36 * 4, kBeta = kG + C * 16, kA = kBeta + C * 4;
  static constexpr int kB = kA + C * 4, kFall = kB + 128, kRows = kFall + C * 4, kBad = kRows + 128 * 8, kBar = kBad + 128, kBytes = kBar + 64;
};
struct Scalars {
  float decay, t, m;  // e^(G_C); what products with T and with M are multiplied by
  int first;          // the first token whose key, gate or step size is not finite (C: none)
  uint32_t odd_q[2];  // a bit for every token whose query is not
};

// Byte offset of 16-byte chunk q of row r, rows of `row` bytes, chunks permuted by r % 8.
__device__ __forceinline__ uint32_t swz(int r, int q, int row) { return r * row + ((q ^ (r & 7)) << 4); }

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Arrives with nothing written that the waiting threads read (they may write what this thread has read).
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_publish(int id, int threads) {
  __threadfence_block();
  bar_arrive(id, threads);
}
// Waits for a phase of `bar`; gives up after a second or so and reports it (the products that are waited for
// have been issued, so this ends long before).
__device__ __forceinline__ void wait_phase(uint64_t* bar, uint32_t phase, int* err) {
#pragma unroll 1
  for (int i = 0; i < (1 << 20); ++i)
    if (mbar_try_wait_sleep(bar, phase, 1000)) return;
  report(err, ERR_WAIT);
}

__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) { return unpack_half2(u); }

// The larger magnitudes of two pairs (a NaN gives way to a number).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 v = __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, __half) {
  const __half2 v = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&a)), __habs2(*reinterpret_cast<const __half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ int clamp_exponent(float x) { return max(-100, min(110, exponent(x))); }

// ---------------------------------------------------------------- preparing a chunk (256 threads)
// Every other 16-byte chunk of row r (keys, then queries) from `raw` to binary16 with the row's exponent taken
// out. x: the factor that brings products back, 2^e / norm; y: a bound of the norm of what that gives. A row that is not
// finite becomes zeros and is noted.
template <typename T, int DK>
__device__ __forceinline__ float2 prepare_row(const uint8_t* raw, uint8_t* to, int r, int half, bool l2norm, float eps,
                                              float scale, Scalars* notes) {
  constexpr int Q = DK / 16;  // 16-byte chunks of half a row
  const uint8_t* const from = raw + r * Smem<DK>::kRow + half * 16;
  uint32_t top = 0u;
#pragma unroll 2
  for (int q = 0; q < Q; ++q) {
    const uint4 x = *reinterpret_cast<const uint4*>(from + 32 * q);
    top = max_abs2(top, max_abs2(max_abs2(x.x, x.y, T()), max_abs2(x.z, x.w, T()), T()), T());
  }
  const float2 both = unpack2(top, T());
  float mx = fmaxf(both.x, both.y);
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  const int e = clamp_exponent(mx);
  const float f = pow2i(-e);
  float ss[2] = {0.f, 0.f};
#pragma unroll 2
  for (int q = 0; q < Q; ++q) {
    const uint4 x = *reinterpret_cast<const uint4*>(from + 32 * q);
    uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = unpack2(u[j], T());
      const float a = v.x * f, b = v.y * f;
      ss[j & 1] = fmaf(a, a, fmaf(b, b, ss[j & 1]));
      u[j] = pack_half2(a, b);
    }
    const int chunk = 2 * q + half;
    *reinterpret_cast<uint4*>(to + (chunk >> 3) * Smem<DK>::kPanel + swz(r, chunk & 7, 128)) =
        make_uint4(u[0], u[1], u[2], u[3]);
  }
  float sum = ss[0] + ss[1];
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  if (!(sum < INFINITY)) {
#pragma unroll 1
    for (int q = half; q < 2 * Q; q += 2)
      *reinterpret_cast<uint4*>(to + (q >> 3) * Smem<DK>::kPanel + swz(r, q & 7, 128)) = make_uint4(0u, 0u, 0u, 0u);
    if (r < C)
      atomicMin(&notes->first, r);
    else
      atomicOr(&notes->odd_q[(r - C) >> 5], 1u << (r & 31));
    return make_float2(0.f, 0.f);
  }
  // 2^e / sqrt(2^2e ss + eps) = 1 / sqrt(ss + 2^-2e eps), with the two factors of 2^-e apart
  float a = pow2i(e);
  if (l2norm) {
    const float y = sum + eps * f * f, h = rsqrtf(y);
    a = h == INFINITY || h == 0.f ? h : fmaf(0.5f * h, fmaf(-y * h, h, 1.0f), h);  // and one step of Newton's
  }
  a = mx == 0.f ? 0.f : scale * a;
  return make_float2(a, 1.01f * fabsf(a) * sum * rsqrtf(fmaxf(sum, 1e-30f)));
}

// Running decays are sums of base-2 logarithms in two binary32 parts, so that the decay from one token to a
// near one is exact whatever came before them in the chunk.
__device__ __forceinline__ float decay_between(float4 later, float4 earlier) {
  return exp2_fast((later.x - earlier.x) + (later.y - earlier.y));
}

// The largest of a warp's values, none negative.
__device__ __forceinline__ float max_of_warp(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// The sum of two numbers in two binary32 parts each, in two parts (the error of the leading sum kept).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  const float s = __fadd_rn(a.x, b.x), t = __fsub_rn(s, a.x);
  const float e = __fadd_rn(__fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t)), __fadd_rn(a.y, b.y));
  const float hi = __fadd_rn(s, e);
  return make_float2(hi, __fsub_rn(e, __fsub_rn(hi, s)));
}

// Two columns of a row of a product over 8: the sum of a[k] b[k][0..1], b's rows ldb apart.
__device__ __forceinline__ float2 row_product(const float* a, const float* b, int ldb) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    const float4 v = *reinterpret_cast<const float4*>(a + k);
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = *reinterpret_cast<const float2*>(b + (k + j) * ldb);
      s.x = fmaf(x[j], y.x, s.x);
      s.y = fmaf(x[j], y.y, s.y);
    }
  }
  return s;
}

// One 16 x 8 tile of a product over K, by a warp, in tf32 parts (the products of two low parts are left out:
// 2^-22): y = sign * a[16 x K] b[K x 8].
template <int K>
__device__ __forceinline__ void tile_product(float* y, int ldy, const float* a, const float* b, int ldb, float sign, int lane) {
  const int g = lane >> 2, c = lane & 3;
  float s[4] = {}, t[4] = {}, u[4] = {};
#pragma unroll
  for (int k = 0; k < K; k += 8) {
    uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) split_tf32(a[(g + 8 * (j & 1)) * LD + k + c + 4 * (j >> 1)], ah[j], al[j]);
#pragma unroll
    for (int j = 0; j < 2; ++j) split_tf32(b[(k + c + 4 * j) * ldb + g], bh[j], bl[j]);
    mma_tf32(t, ah, bl);
    mma_tf32(u, al, bh);
    mma_tf32(s, ah, bh);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = sign * (s[j] + (t[j] + u[j]));
  *reinterpret_cast<float2*>(y + g * ldy + 2 * c) = make_float2(s[0], s[1]);
  *reinterpret_cast<float2*>(y + (g + 8) * ldy + 2 * c) = make_float2(s[2], s[3]);
}

// (I + X)^-1 in the place of X, lower triangle by blocks: the lower left of [[A, 0], [B, D]]^-1 is -D^-1 B A^-1.
__device__ __forceinline__ void invert(float* X, float* Y, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  if (warp < 4) {
    // 8 x 8 on the diagonal by substitution, a column each lane; a warp has the two blocks of its 16 rows
    if (lane < 16) {
      const int o = 16 * warp + (lane & 8), c = lane & 7;
      const float* const l = X + o * LD + o;
      float y[8], x[28];
#pragma unroll
      for (int i = 1; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < i; ++j) x[i * (i - 1) / 2 + j] = -l[i * LD + j];
      __syncwarp(0xffffu);  // every lane has read its block
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = i == c ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < 7; ++j)  // y[j] is known; take it out of the rows below
#pragma unroll
        for (int i = j + 1; i < 8; ++i) y[i] = fmaf(x[i * (i - 1) / 2 + j], y[j], y[i]);
#pragma unroll
      for (int i = 0; i < 8; ++i) X[(o + i) * LD + o + c] = y[i];
    }
    __syncwarp();
    const int o = 16 * warp, row = lane >> 2, col = 2 * (lane & 3);
    float* const y = Y + warp * 8 * 12;
    *reinterpret_cast<float2*>(y + row * 12 + col) = row_product(X + (o + 8 + row) * LD + o, X + o * LD + o + col, LD);
    *reinterpret_cast<float2*>(X + (o + row) * LD + o + 8 + col) = make_float2(0.f, 0.f);
    __syncwarp();
    const float2 t = row_product(X + (o + 8 + row) * LD + o + 8, y + col, 12);
    *reinterpret_cast<float2*>(X + (o + 8 + row) * LD + o + col) = make_float2(-t.x, -t.y);
  }
  bar_sync(kBarAux, kAux);
  {  // 16 and 16: a pair of blocks by two warps; the others clear what lies above them
    const int pair = warp >> 1 & 1, o = 32 * pair, col = 8 * (warp & 1);
    float* const y = Y + pair * 16 * 20 + col;
    if (warp < 4) {
      tile_product<16>(y, 20, X + (o + 16) * LD + o, X + o * LD + o + col, LD, 1.f, lane);
    } else {
      const int x = tid - 128, row = (x & 63) >> 2;
      *reinterpret_cast<float4*>(X + (32 * (x >> 6) + row) * LD + 32 * (x >> 6) + 16 + 4 * (x & 3)) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    bar_sync(kBarAux, kAux);
    if (warp < 4) tile_product<16>(X + (o + 16) * LD + o + col, LD, X + (o + 16) * LD + o + 16, y, 20, -1.f, lane);
  }
  bar_sync(kBarAux, kAux);
  {  // 32 and 32: a tile each warp
    const int row = 16 * (warp & 1), col = 8 * (warp >> 1);
    tile_product<32>(Y + row * 36 + col, 36, X + (32 + row) * LD, X + col, LD, 1.f, lane);
    bar_sync(kBarAux, kAux);
    tile_product<32>(X + (32 + row) * LD + col, LD, X + (32 + row) * LD + 32, Y + col, 36, -1.f, lane);
  }
  bar_sync(kBarAux, kAux);
}

// next: asks for this chunk's values and the next one's rows, once this one's have been read. gates: this thread's part of the chunk's
// decays and gates (one warp, while the product runs).
template <typename T, int DK, typename Next, typename Gates>
__device__ __forceinline__ void prepare_chunk(const DeltaRun& r, uint8_t* smem, uint8_t* stage, int tid, uint32_t tmem,
                                              uint64_t* bar, uint32_t phase, Next&& next, Gates&& gates) {
  using M = Smem<DK>;
  const fmoe_delta_desc& d = r.d;
  const int warp = tid >> 5;
  float* const L = reinterpret_cast<float*>(smem + M::kL);
  float4* const G = reinterpret_cast<float4*>(smem + M::kG);  // decay (two parts), key's factor
  const float* const beta = reinterpret_cast<const float*>(smem + M::kBeta);
  float* const qb = reinterpret_cast<float*>(smem + M::kA);
  float* const norms = reinterpret_cast<float*>(smem + M::kB);  // keys', queries' largest norms; T's entries
  Scalars* const scalars = reinterpret_cast<Scalars*>(stage + M::kEnd);
  {
    const int row = tid >> 1;
    const float2 a = prepare_row<T, DK>(smem + M::kRaw, stage + M::kKQ, row, tid & 1, d.l2norm, d.eps, row < C ? 1.0f : d.scale, scalars);
    if (!(tid & 1)) *(row < C ? &G[row].z : qb + row - C) = a.x;
    const float top = max_of_warp(a.y);
    if ((tid & 31) == 0) norms[warp] = top;
  }
  fence_proxy_async();
  tc_fence_before();  // the last chunk's loads from these columns
  bar_sync(kBarAux, kAux);
  if (tid == 0) {
    tc_fence_after();
    const uint32_t kq = smem_u32(stage + M::kKQ);
#pragma unroll
    for (int k = 0; k < DK / 16; ++k) {
      const uint64_t x = smem_operand(kq + (k >> 2) * M::kPanel + (k & 3) * 32);
      tc_mma_ss(tmem + kColL, x, x, tc_shape(C), k > 0);
    }
    tc_commit(bar);
  }
  __syncwarp();
  next();
  if (warp == 7) gates();
  wait_phase(bar, phase, r.err);
  tc_fence_after();
  bar_sync(kBarAux, kAux);

  // ---- tensor memory's rows 0-63 are L's, 64-127 M's; warps 0-3 take columns 0-31, warps 4-7 the others, which
  // are zeros in rows below 32
  {
    const int quarter = warp & 3, b = warp >> 2, i = 32 * (quarter & 1) + (tid & 31), limit = quarter < 2 ? i : i + 1;
    const bool any = b <= (quarter & 1);
    const float4 gi = G[i];
    float f;
    if (quarter < 2) {
      f = beta[i] * gi.z;
    } else {
      // |M_ij| is at most the largest of the queries' norms times that of the keys'
      const float4 nk = *reinterpret_cast<const float4*>(norms), nq = *reinterpret_cast<const float4*>(norms + 4);
      const int e = clamp_exponent(fmaxf(fmaxf(nk.x, nk.y), fmaxf(nk.z, nk.w)) *
                                   fmaxf(fmaxf(nq.x, nq.y), fmaxf(nq.z, nq.w))) + 1 - kTop;
      f = qb[i] * pow2i(-e);
      if (b == 0) {
        reinterpret_cast<float*>(stage + M::kOut)[i] = qb[i] * exp2_fast(gi.x);
        if (i == 0) scalars->m = pow2i(e);
      }
    }
    if (any || quarter >= 2) {
#pragma unroll 1
      for (int c0 = 32 * b; c0 < 32 * b + 32; c0 += 16) {
        uint32_t v[16];
        if (any) {
          tc_load16(v, tmem + (uint32_t)(quarter * 32 << 16) + kColL + c0);
          tc_wait_load();
        }
        // The decay from column to row is that to the end of the column's 16 tokens, which multiplies the key's
        // factor already, times that from there to the row: unless it falls too steeply inside the 16.
        const float4 g16 = G[c0 + 15];
        const float4* const fall = reinterpret_cast<const float4*>(smem + M::kFall) + (c0 >> 2);
        if (G[c0].x - g16.x < 40.f && fabsf(f) < 1e18f) {
          const float fi = f * decay_between(gi, g16);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 t = fall[j >> 2];
            v[j] = c0 + j < limit ? __float_as_uint(fi * t.x * __uint_as_float(v[j])) : 0u;
            v[j + 1] = c0 + j + 1 < limit ? __float_as_uint(fi * t.y * __uint_as_float(v[j + 1])) : 0u;
            v[j + 2] = c0 + j + 2 < limit ? __float_as_uint(fi * t.z * __uint_as_float(v[j + 2])) : 0u;
            v[j + 3] = c0 + j + 3 < limit ? __float_as_uint(fi * t.w * __uint_as_float(v[j + 3])) : 0u;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float4 gj = G[c0 + j];
            v[j] = c0 + j < limit ? __float_as_uint((f * gj.z) * decay_between(gi, gj) * __uint_as_float(v[j])) : 0u;
          }
        }
        if (quarter < 2) {
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<uint4*>(L + i * LD + c0 + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              h[j] = pack_half2(__uint_as_float(v[8 * q + 2 * j]), __uint_as_float(v[8 * q + 2 * j + 1]));
            const uint32_t at = swz(i, (c0 >> 3) + q, 128);
            *reinterpret_cast<uint4*>(stage + M::kM + at) = make_uint4(h[0], h[1], h[2], h[3]);
            if (std::is_same<T, __half>::value) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                h[j] = rest_half2(__uint_as_float(v[8 * q + 2 * j]), __uint_as_float(v[8 * q + 2 * j + 1]), h[j]);
              *reinterpret_cast<uint4*>(stage + M::kMl + at) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
      }
    }
  }
  bar_sync(kBarAux, kAux);
  invert(L, reinterpret_cast<float*>(smem + M::kY), tid);

  // ---- T, its columns times beta, in two binary16 parts, a quarter of a row each thread; the tokens' factors
  {
    const int row = tid >> 2, part = tid & 3;
    float v[16], top = 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 a = part > 1 && row < 32 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                            : *reinterpret_cast<const float4*>(L + row * LD + 16 * part + j);
      const float4 b = *reinterpret_cast<const float4*>(beta + 16 * part + j);
      v[j] = a.x * b.x, v[j + 1] = a.y * b.y, v[j + 2] = a.z * b.z, v[j + 3] = a.w * b.w;
      top = fmaxf(top, fmaxf(fmaxf(fabsf(v[j]), fabsf(v[j + 1])), fmaxf(fabsf(v[j + 2]), fabsf(v[j + 3]))));
    }
    const float4 last = G[C - 1], g = G[row];
    const float w = decay_between(last, g) * g.z;
    top = max_of_warp(top);
    if ((tid & 31) == 0) norms[8 + warp] = top;
    bar_sync(kBarAux, kAux);
    const float4 ta = *reinterpret_cast<const float4*>(norms + 8), tb = *reinterpret_cast<const float4*>(norms + 12);
    const int e = clamp_exponent(fmaxf(fmaxf(fmaxf(ta.x, ta.y), fmaxf(ta.z, ta.w)),
                                       fmaxf(fmaxf(tb.x, tb.y), fmaxf(tb.z, tb.w)))) - kTop;
    const float s = pow2i(-e);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t h[4], l[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[8 * q + 2 * j] * s, b = v[8 * q + 2 * j + 1] * s;
        h[j] = pack_half2(a, b);
        l[j] = rest_half2(a, b, h[j]);
      }
      const uint32_t at = swz(row, 2 * part + q, 128);
      *reinterpret_cast<uint4*>(stage + M::kTh + at) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(stage + M::kTl + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
    if (part == 0) {
      reinterpret_cast<float*>(stage + M::kCa)[row] = exp2_fast(g.x) * g.z;
      reinterpret_cast<float*>(stage + M::kW)[row] = w;
      if (row == 0) {
        scalars->decay = exp2_fast(last.x), scalars->t = pow2i(e);
      }
    }
  }
  fence_proxy_async();
  bar_sync(kBarAux, kAux);  // the next chunk's decays and gates may come
}

template <typename T, int DK>
__device__ __forceinline__ void prepare_all(const DeltaRun& r, uint8_t* smem, int seq, int head, int begin, int end,
                                            uint32_t tmem, uint64_t* bar) {
  using M = Smem<DK>;
  const fmoe_delta_desc& d = r.d;
  const int tid = threadIdx.x - kChain, lane = tid & 31, chunks = (end - begin + C - 1) / C;
  const int hk = head / (d.heads_v / d.heads_k);
  const T* const k = static_cast<const T*>(d.k.ptr) + hk * d.k.head_stride;
  const T* const q = static_cast<const T*>(d.q.ptr) + hk * d.q.head_stride;
  const T* const v = static_cast<const T*>(d.v.ptr) + head * d.v.head_stride;
  // Rows behind the sequence's end are zeros: no key, no query, no gate.
  auto copy16_or_zero = [&](uint32_t at, const T* from, int t) {
    if (t < end)
      copy16(at, from);
    else
      asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
  };
  auto copy_raw = [&](int t0) {  // keys by the first half of the threads, queries by the others
    constexpr int kLog = DK == 64 ? 3 : 4, kStep = 128 >> kLog;  // chunks of a row, rows at a time
    const int half = tid >> 7, row = (tid & 127) >> kLog, col = tid & ((1 << kLog) - 1);
    const int64_t stride = half ? d.q.token_stride : d.k.token_stride;
    const T* from = (half ? q : k) + (t0 + row) * stride + col * 8;
    uint32_t at = smem_u32(smem + M::kRaw) + (half * C + row) * M::kRow + col * 16;
#pragma unroll 4
    for (int x = 0; x < C; x += kStep) {
      copy16_or_zero(at, from, t0 + row + x);
      from += kStep * stride;
      at += kStep * M::kRow;
    }
    copy_commit();
  };
  auto copy_values = [&](uint32_t to, int t0) {
    const int log = d.dim_v == 64 ? 3 : 4, step = 256 >> log, row = tid >> log;
    const T* from = v + (t0 + row) * d.v.token_stride + (tid - (row << log)) * 8;
    uint32_t at = to + tid * 16;
#pragma unroll 2
    for (int x = 0; x < C; x += step) {
      copy16_or_zero(at, from, t0 + row + x);
      from += step * d.v.token_stride;
      at += kAux * 16;
    }
    copy_commit();
  };
  float gn[2], bn[2];
  auto fetch_gates = [&](int t0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = t0 + 2 * lane + j;
      gn[j] = t < end ? d.g[t * d.gate_stride + head] : 0.f;
      bn[j] = t < end ? d.beta[t * d.gate_stride + head] : 0.f;
    }
  };
  copy_raw(begin);
  if (tid >= kAux - 32) fetch_gates(begin);
#pragma unroll 1
  for (int n = 0; n < chunks; ++n) {
    uint8_t* const stage = smem + (n & 1) * M::kStage;
    const int t0 = begin + n * C;
    if (n >= 2) bar_sync(kBarFree + (n & 1), kThreads);
    Scalars* const notes = reinterpret_cast<Scalars*>(stage + M::kEnd);
    if (tid == 0) notes->first = C, notes->odd_q[0] = notes->odd_q[1] = 0u;
    copy_wait<0>();  // this chunk's keys and queries
    bar_sync(kBarAux, kAux);
    auto next = [&]() {
      copy_values(smem_u32(stage + M::kV), t0);
      if (n + 1 < chunks)
        copy_raw(t0 + C);
      else
        copy_commit();
    };
    auto gates = [&]() {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!(gn[j] <= 88.72f && fabsf(bn[j]) < INFINITY)) {  // e^88.73 is infinite
          gn[j] = bn[j] = 0.f;
          atomicMin(&notes->first, 2 * lane + j);
        }
        gn[j] *= kLog2e;
        if (gn[j] < -300.f) gn[j] = -300.f;  // nothing is left below 2^-149
      }
      float2 sum = add2(make_float2(gn[0], 0.f), make_float2(gn[1], 0.f));
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const float2 o = make_float2(__shfl_up_sync(0xffffffffu, sum.x, m), __shfl_up_sync(0xffffffffu, sum.y, m));
        if (lane >= m) sum = add2(sum, o);
      }
      float4* const to = reinterpret_cast<float4*>(smem + M::kG) + 2 * lane;
      *reinterpret_cast<float2*>(to) = add2(sum, make_float2(-gn[1], 0.f));
      *reinterpret_cast<float2*>(to + 1) = sum;
      const float2 first = add2(sum, make_float2(-gn[1], 0.f));
      const float4 end16 = make_float4(__shfl_sync(0xffffffffu, sum.x, lane | 7), __shfl_sync(0xffffffffu, sum.y, lane | 7), 0.f, 0.f);
      reinterpret_cast<float2*>(smem + M::kFall)[lane] =
          make_float2(to[0].z * decay_between(end16, make_float4(first.x, first.y, 0.f, 0.f)),
                      to[1].z * decay_between(end16, make_float4(sum.x, sum.y, 0.f, 0.f)));
      reinterpret_cast<float2*>(smem + M::kBeta)[lane] = make_float2(bn[0], bn[1]);
      if (n + 1 < chunks) fetch_gates(t0 + C);
    };
    prepare_chunk<T, DK>(r, smem, stage, tid, tmem, bar, n & 1, next, gates);
    copy_wait<1>();  // the values; the next rows may still be on their way
    bar_publish(kBarFull + (n & 1), kThreads);
  }
  copy_wait<0>();
  // the chain and the outputs free every stage: the last two barriers are met here
  for (int n = max(chunks, 2); n < chunks + 2; ++n) bar_sync(kBarFree + (n & 1), kThreads);
}

// ---------------------------------------------------------------- the chain (128 threads, a row each)
// The larger of two, a NaN where either is one.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// 32 values times f as the parts of a left operand: 16 columns high, 16 low (where wanted).
template <bool LOW>
__device__ __forceinline__ void store_parts(uint32_t to, const uint32_t (&x)[32], float f) {
  uint32_t h[16], l[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float a = __uint_as_float(x[2 * j]) * f, c = __uint_as_float(x[2 * j + 1]) * f;
    h[j] = pack_half2(a, c);
    if (LOW) l[j] = rest_half2(a, c, h[j]);
  }
  tc_store16(to, h);
  if (LOW) tc_store16(to + 16, l);
}
// 64 columns of values by their parts.
__device__ __forceinline__ void replace_by_parts(uint32_t at, float f) {
#pragma unroll 1
  for (int b = 0; b < C; b += 32) {
    uint32_t p[32];
    tc_load32(p, at + b);
    tc_wait_load();
    store_parts<true>(at + b, p, f);
  }
}

template <typename T, int DK>
__device__ __forceinline__ void chain(const DeltaRun& r, uint8_t* smem, int seq, int head, int slot, int chunks,
                                      uint32_t tmem, uint64_t* bar, uint64_t* qs_bar, uint64_t* out_bar) {
  using M = Smem<DK>;
  constexpr bool kLow = std::is_same<T, __half>::value;  // low parts for the outputs too
  const fmoe_delta_desc& d = r.d;
  const int row = threadIdx.x;
  const bool real = row < d.dim_v;  // rows behind dim_v (64) carry zeros
  const uint32_t lanes = tmem + (uint32_t)((row & ~31) << 16);
  float* const state = d.state + slot * d.state_stride + (int64_t)head * DK * d.dim_v + row;
  float2* const scales = reinterpret_cast<float2*>(smem + M::kRows);
  // The state is S times `unit`, a power of two that keeps S inside binary16's range (2^-40 at least, so that values of
  // 2^80 may still follow; binary16's last place is then 2^-65); what the last chunk left to be done to S is
  // S = grow * S + increment.
  float unit = 1.f, grow = 1.f, top = 0.f;
  {
    const bool load = real && !(r.fresh && r.fresh[seq]);
    const uint32_t zero[16] = {};
#pragma unroll 1
    for (int b = 0; b < DK; b += 16) {
      uint32_t v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float x = load ? state[(int64_t)(b + j) * d.dim_v] : 0.f;
        v[j] = __float_as_uint(x);
        top = fmaxf(top, fabsf(x));
      }
      tc_store16(lanes + kColS + b, v);
      tc_store16(lanes + kColA + b, zero);
    }
    tc_wait_store();
    if (top > 0.f) {
      const int e = max(clamp_exponent(top) - 12, -40);
      unit = pow2i(e);
      grow = pow2i(-e);
    }
  }
  uint32_t phase = 0;
  auto done = [&]() {
    wait_phase(bar, phase, r.err);
    phase ^= 1;
    tc_fence_after();
  };
  auto ready = [&]() {  // every thread's operand rows are written
    tc_wait_store();
    tc_fence_before();
    bar_sync(kBarMain, 128);
  };
#pragma unroll 1
  for (int n = 0; n < chunks; ++n) {
    uint8_t* const stage = smem + (n & 1) * M::kStage;
    const uint32_t st = smem_u32(stage);
    const float* const ca = reinterpret_cast<const float*>(stage + M::kCa);
    const float* const w = reinterpret_cast<const float*>(stage + M::kW);
    const Scalars* const scalars = reinterpret_cast<const Scalars*>(stage + M::kEnd);
    // ---- S, and its parts
    top = 0.f;
#pragma unroll 1
    for (int b = 0; b < DK; b += 32) {
      uint32_t v[32], p[32];
      tc_load32(v, lanes + kColS + b);
      tc_load32(p, lanes + kColA + b);
      tc_wait_load();
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float x = fmaf(grow, __uint_as_float(v[j]), __uint_as_float(p[j]));
        top = fmaxf(top, fabsf(x));
        v[j] = __float_as_uint(x);
      }
      tc_store32(lanes + kColS + b, v);
      store_parts<true>(lanes + kColA + b, v, 1.f);
    }
    bar_sync(kBarFull + (n & 1), kThreads);
    if (n > 0) bar_sync(kBarOut, 256);
    ready();
    // ---- [K S | Q S]: high parts, low parts with K; low parts with Q where the output is that exact
    if (threadIdx.x == 0) {
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < DK / 16; ++k)
        tc_mma_ts(tmem + kColP, tmem + kColA + 32 * (k >> 1) + 8 * (k & 1),
                  smem_operand(st + M::kKQ + (k >> 2) * M::kPanel + (k & 3) * 32), tc_shape(2 * C), k > 0);
#pragma unroll 2
      for (int k = 0; k < DK / 16; ++k)
        tc_mma_ts(tmem + kColP, tmem + kColA + 32 * (k >> 1) + 8 * (k & 1) + 16,
                  smem_operand(st + M::kKQ + (k >> 2) * M::kPanel + (k & 3) * 32), tc_shape(kLow ? 2 * C : C), true);
      tc_commit(bar);
      tc_commit(qs_bar);
    }
    __syncwarp();
    done();
    // ---- the right-hand side v - e^G K S (beta is in T's columns)
    float mx = 0.f;
#pragma unroll 1
    for (int b = 0; b < C; b += 32) {
      uint32_t p[32];
      float y[32];
      tc_load32(p, lanes + kColP + b);
      const T* const v = reinterpret_cast<const T*>(stage + M::kV) + (real ? row : 0) + b * d.dim_v;
#pragma unroll
      for (int j = 0; j < 32; ++j) y[j] = to_f32(v[j * d.dim_v]);
      tc_wait_load();
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 t = *reinterpret_cast<const float4*>(ca + b + j);
        const float a[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float z = fmaf(-unit * a[i], __uint_as_float(p[j + i]), y[j + i]);
          mx = max_or_nan(mx, fabsf(z));
          p[j + i] = __float_as_uint(z);
        }
      }
      tc_store32(lanes + kColP + b, p);
    }
    tc_wait_store();
    int odd = scalars->first;  // the first token of this row that is not finite
    if (__any_sync(0xffffffffu, odd < C || !(mx < INFINITY))) {
      mx = 0.f;
#pragma unroll 1
      for (int b = 0; b < C; b += 32) {
        uint32_t p[32];
        tc_load32(p, lanes + kColP + b);
        tc_wait_load();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float z = fabsf(__uint_as_float(p[j]));
          if (!(z < INFINITY)) odd = min(odd, b + j);
          if (b + j >= odd) p[j] = 0u;
          mx = fmaxf(mx, fabsf(__uint_as_float(p[j])));
        }
        tc_store32(lanes + kColP + b, p);
      }
      tc_wait_store();
    }
    smem[M::kBad + row] = (uint8_t)odd;
    int e = clamp_exponent(mx) - kTop;
    const float back = pow2i(e) / unit;
    replace_by_parts(lanes + kColP, pow2i(-e));
    ready();
    // ---- U = T times it
    if (threadIdx.x == 0) {
      tc_fence_after();
#pragma unroll
      for (int part = 0; part < 3; ++part)  // high x high, low x high, high x low
#pragma unroll
        for (int k = 0; k < C / 16; ++k)
          tc_mma_ts(tmem + kColU, tmem + kColP + (part == 1 ? 16 : 0) + 32 * (k >> 1) + 8 * (k & 1),
                    smem_operand(st + (part == 2 ? M::kTl : M::kTh) + k * 32), tc_shape(C), part + k > 0);
      tc_commit(bar);
    }
    __syncwarp();
    done();
    float sum = 0.f;  // of what the tokens add to the state, but for the keys (below 2)
    mx = 0.f;
    {  // from here on in units
      const float f = back * scalars->t;
#pragma unroll 1
      for (int b = 0; b < C; b += 32) {
        uint32_t p[32];
        tc_load32(p, lanes + kColU + b);
        tc_wait_load();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 t = *reinterpret_cast<const float4*>(w + b + j);
          const float a[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = __uint_as_float(p[j + i]) * f;
            mx = fmaxf(mx, fabsf(u));
            sum += fabsf(u * a[i]);
            p[j + i] = __float_as_uint(u);
          }
        }
        tc_store32(lanes + kColU + b, p);
      }
      tc_wait_store();
    }
    // ---- M U, for the outputs, in the place of Q S once that is taken
    e = clamp_exponent(mx) - kTop;
    scales[row] = make_float2(unit, unit * pow2i(e));
    {
      const float f = pow2i(-e);
#pragma unroll 1
      for (int b = 0; b < C; b += 32) {
        uint32_t p[32];
        tc_load32(p, lanes + kColU + b);
        tc_wait_load();
        store_parts<kLow>(lanes + kColP + b, p, f);
      }
    }
    bar_sync(kBarTaken, 256);
    ready();
    if (threadIdx.x == 0) {
      tc_fence_after();
#pragma unroll
      for (int part = 0; part < (kLow ? 3 : 1); ++part)  // high x high, low x high, high x low
#pragma unroll
        for (int k = 0; k < C / 16; ++k)
          tc_mma_ts(tmem + kColO, tmem + kColP + (part == 1 ? 16 : 0) + 32 * (k >> 1) + 8 * (k & 1),
                    smem_operand(st + (part == 2 ? M::kMl : M::kM) + k * 32), tc_shape(C), part + k > 0);
      tc_commit(out_bar);
    }
    __syncwarp();
    bar_publish(kBarScales, 256);
    // ---- the state's increment (e^(G_C - G) K)^T U in the unit of the next chunk: this one, unless what S can
    // come to (keys are below 2) leaves binary16's range or falls far below it
    grow = scalars->decay;
    float f = 1.f;
    {
      const float most = fmaf(grow, top, 2.f * sum);
      if (!(most <= 32768.f && most >= 128.f) && most > 0.f) {
        const int now = exponent(unit), shift = max(-40, min(110, now + clamp_exponent(most) - 12)) - now;
        f = pow2i(max(-126, min(126, -shift)));
        unit = pow2i(now + shift);
        grow *= f;
      }
      if (odd < C) grow = NAN;
    }
#pragma unroll 1
    for (int b = 0; b < C; b += 32) {
      uint32_t p[32];
      tc_load32(p, lanes + kColU + b);
      tc_wait_load();
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 t = *reinterpret_cast<const float4*>(w + b + j);
        p[j] = __float_as_uint(__uint_as_float(p[j]) * t.x);
        p[j + 1] = __float_as_uint(__uint_as_float(p[j + 1]) * t.y);
        p[j + 2] = __float_as_uint(__uint_as_float(p[j + 2]) * t.z);
        p[j + 3] = __float_as_uint(__uint_as_float(p[j + 3]) * t.w);
      }
      store_parts<true>(lanes + kColU + b, p, f);
    }
    ready();
    if (threadIdx.x == 0) {
      tc_fence_after();
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < C / 16; ++k)
          tc_mma_ts(tmem + kColA, tmem + kColU + part * 16 + 32 * (k >> 1) + 8 * (k & 1),
                    smem_operand(st + M::kKQ + k * 2048, M::kPanel), tc_shape(DK, true), part + k > 0);
      tc_commit(bar);
    }
    __syncwarp();
    done();
    bar_arrive(kBarFree + (n & 1), kThreads);
  }
#pragma unroll 1
  for (int b = 0; b < DK; b += 32) {
    uint32_t v[32], p[32];
    tc_load32(v, lanes + kColS + b);
    tc_load32(p, lanes + kColA + b);
    tc_wait_load();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (real) state[(int64_t)(b + j) * d.dim_v] = unit * fmaf(grow, __uint_as_float(v[j]), __uint_as_float(p[j]));
  }
}

// ---------------------------------------------------------------- the outputs (128 threads, a column each)
template <typename T, int DK>
__device__ __forceinline__ void outputs(const DeltaRun& r, uint8_t* smem, int head, int begin, int end, uint32_t tmem,
                                        uint64_t* qs_bar, uint64_t* bar) {
  using M = Smem<DK>;
  const fmoe_delta_desc& d = r.d;
  const int row = threadIdx.x - kChain - kAux, chunks = (end - begin + C - 1) / C;
  const uint32_t lanes = tmem + (uint32_t)((row & ~31) << 16);
  T* const out = static_cast<T*>(d.out.ptr) + head * d.out.head_stride + begin * d.out.token_stride;
  const int64_t stride = d.out.token_stride;
#pragma unroll 1
  for (int n = 0; n < chunks; ++n) {
    const uint8_t* const stage = smem + (n & 1) * M::kStage;
    const float* const oq = reinterpret_cast<const float*>(stage + M::kOut);
    T* const values = reinterpret_cast<T*>(smem + (n & 1) * M::kStage + M::kV);
    bar_sync(kBarFull + (n & 1), kThreads);
    wait_phase(qs_bar, n & 1, r.err);
    tc_fence_after();
    uint32_t x[2][32];
    tc_load32(x[0], lanes + kColO);
    tc_load32(x[1], lanes + kColO + 32);
    tc_wait_load();
    tc_fence_before();
    bar_arrive(kBarTaken, 256);
    bar_sync(kBarScales, 256);
    const float2 sc = reinterpret_cast<const float2*>(smem + M::kRows)[row];
    const Scalars* const notes = reinterpret_cast<const Scalars*>(stage + M::kEnd);
    const float fm = sc.y * notes->m;
    const int odd = smem[M::kBad + row];
    const uint32_t odd_q[2] = {notes->odd_q[0], notes->odd_q[1]};
    wait_phase(bar, n & 1, r.err);
    tc_fence_after();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t y[32];
      tc_load32(y, lanes + kColO + 32 * b);
      tc_wait_load();
      if (b == 1) {
        tc_fence_before();
        if (n + 1 < chunks) bar_arrive(kBarOut, 256);
      }
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 t = *reinterpret_cast<const float4*>(oq + 32 * b + j);
        const float a[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[b][j + i] = __float_as_uint(fmaf(a[i] * sc.x, __uint_as_float(x[b][j + i]), fm * __uint_as_float(y[j + i])));
      }
    }
    if (odd < C || (odd_q[0] | odd_q[1])) {
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (j >= odd || (odd_q[j >> 5] >> (j & 31) & 1u)) x[j >> 5][j & 31] = 0x7fffffffu;  // NaN
    }
    // rows of tokens in the place of the values, which the chain has taken; then out in whole 16 bytes
    {
      T* to = values + row;
      if (row < d.dim_v) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
          *to = from_f32<T>(__uint_as_float(x[j >> 5][j & 31]));
          to += d.dim_v;
        }
      }
    }
    bar_sync(kBarRows, kOutputs);
    {
      const int log = d.dim_v == 64 ? 3 : 4, left = min(C, end - begin - n * C);
#pragma unroll 2
      for (int i = row; i < left << log; i += kOutputs) {
        const int token = i >> log, col = 8 * (i - (token << log));
        *reinterpret_cast<uint4*>(out + ((int64_t)n * C + token) * stride + col) =
            *reinterpret_cast<const uint4*>(values + i * 8);
      }
    }
    bar_arrive(kBarFree + (n & 1), kThreads);
  }
}

template <typename T, int DK>
__global__ void __launch_bounds__(kThreads, 1) delta_chunk(const DeltaRun r) {
  using M = Smem<DK>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const fmoe_delta_desc& d = r.d;
  const int head = blockIdx.x % d.heads_v, seq = blockIdx.x / d.heads_v;
  const int begin = r.cu[seq], end = r.cu[seq + 1];
  if (begin < 0 || end < begin || end > r.n_tokens) {
    if (threadIdx.x == 0) report(r.err, ERR_LENGTH);
    return;
  }
  if (begin == end) return;
  const int slot = d.slots ? d.slots[seq] : seq;
  if (slot < 0 || slot >= d.n_slots) {
    if (threadIdx.x == 0 && slot >= 0) report(r.err, ERR_SLOT);
    return;
  }
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + M::kBar);  // products: the chain, Q S, preparing, M U
  uint32_t* const base = reinterpret_cast<uint32_t*>(bars + 4);
  if (threadIdx.x < 32) tc_alloc(base);
  if (threadIdx.x == 32) {
    for (int i = 0; i < 4; ++i) mbar_init(bars + i, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // All columns are this block's: they begin at 0, which the products' addresses below are made from.
  constexpr uint32_t tmem = 0;
  // The registers of the launch (128 a thread) are dealt out again: 152 + 2 * 112 + 136 = 4 * 128.
  if (threadIdx.x < kChain) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    chain<T, DK>(r, smem, seq, head, slot, (end - begin + C - 1) / C, tmem, bars, bars + 1, bars + 3);
  } else if (threadIdx.x < kChain + kAux) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    prepare_all<T, DK>(r, smem, seq, head, begin, end, tmem, bars + 2);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    outputs<T, DK>(r, smem, head, begin, end, tmem, bars + 1, bars + 3);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) tc_free(tmem);
}

template <typename T, int DK>
cudaError_t run(const DeltaRun& r, cudaStream_t st) {
  const auto kernel = delta_chunk<T, DK>;
  constexpr int kBytes = Smem<DK>::kBytes;
  static_assert(kBytes <= 232448, "shared memory of a block");
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)r.n * (unsigned)r.d.heads_v, kThreads, kBytes, st>>>(r);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaRun& r, cudaStream_t st) {
  if (r.d.dtype == FMOE_BF16) return r.d.dim_k == 64 ? run<__nv_bfloat16, 64>(r, st) : run<__nv_bfloat16, 128>(r, st);
  return r.d.dim_k == 64 ? run<__half, 64>(r, st) : run<__half, 128>(r, st);
}

}  // namespace fmoe
