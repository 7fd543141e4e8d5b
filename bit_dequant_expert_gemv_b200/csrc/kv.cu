// kv.cu — appending rotated keys and values to the paged 4-bit cache, and reading rows back.
//
// A warp takes a token, or some of its rows: it computes the token's cosines and sines (binary64, so that
// positions of a long context keep every bit of their angle), keeps those of its columns in registers, and goes
// through the query rows, two loads in flight, then the key and value rows. A lane holds dim/32 neighbouring
// columns; a rotated column's partner is beside it or in another lane; the 64 columns that share a scale and a
// bias lie in 2048/dim neighbouring lanes, whose minimum and maximum are taken by shuffles. The quantiser is
// fmoe_pack's, IEEE-rounded binary32 operations, but that the range is multiplied by 1/15 for the scale.
// At many tokens bytes should bound it (the rows in, rotated queries and codes out), and instructions come
// close: 4750 of a warp for a token of 32 query and 2 kv heads of 256, its angles among them. At few tokens latency does:
// there each row has a warp. Measured, appending and reading back: 8192 such tokens 76 and 10 us, half the copy rate,
// the appending issuing in 52 % of the cycles; 32 tokens of 32 and 4 heads of 128 6.8 us for both, two launches.
#include "api.h"
#include "mixer.h"

namespace fmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Place {
  uint8_t* block;  // of head 0
  int at;          // position in the page
};

// The page of a token, or a null block: padding, or an index out of range (reported).
__device__ __forceinline__ Place place_of(const fmoe_kv_cache& c, const int32_t* positions, const int32_t* seq,
                                          int t, size_t block, int* err, bool tell) {
  const int pos = positions[t];
  if (pos < 0) return {nullptr, 0};
  const int i = seq ? seq[t] : t, j = pos / c.page_size;
  if (i < 0 || i >= c.n_seqs || j >= c.max_pages) {
    if (tell) report(err, ERR_POSITION);
    return {nullptr, 0};
  }
  const int page = c.page_table[i * c.table_stride + j];
  if (page < 0 || page >= c.n_pages) {
    if (tell) report(err, ERR_PAGE);
    return {nullptr, 0};
  }
  return {static_cast<uint8_t*>(c.pages) + (size_t)page * c.heads * block, pos - j * c.page_size};
}

// The smaller and the larger of two, a NaN where either is one.
__device__ __forceinline__ float min_or_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Codes of `N` columns of one lane, and the group's scale and bias word. A NaN among the 64 makes minimum and maximum
// NaN in every lane, an infinity the scale infinite: either way all 64 are read back as no numbers.
template <int N>
__device__ __forceinline__ uint32_t quantise(const float* x, uint32_t* sb) {
  constexpr int kLanes = 64 / N;  // lanes of a group
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    mn = min_or_nan(mn, x[i]);
    mx = max_or_nan(mx, x[i]);
  }
#pragma unroll
  for (int m = 1; m < kLanes; m <<= 1) {
    mn = min_or_nan(mn, __shfl_xor_sync(0xffffffffu, mn, m));
    mx = max_or_nan(mx, __shfl_xor_sync(0xffffffffu, mx, m));
  }
  // a product, not a division: the nearest bf16 to a fifteenth of the range but where that is within 2^-22 of the
  // middle of two (one group in 400 of binary16 rows is exactly there), and then one of the two all the same. Elementwise
  // programs on a GPU that divide by the constant 15 multiply so too, and rows that they quantised hold the same codes;
  // fmoe_pack, which converts weights once, divides.
  const __nv_bfloat16 sbf = __float2bfloat16_rn(__fmul_rn(__fsub_rn(mx, mn), 1.0f / 15.0f));
  const __nv_bfloat16 zbf = __float2bfloat16_rn(mn);
  const float s = __bfloat162float(sbf), z = __bfloat162float(zbf);
  *sb = (uint32_t)__bfloat16_as_ushort(sbf) | (uint32_t)__bfloat16_as_ushort(zbf) << 16;
  uint32_t codes = 0;
  if (s != 0.0f) {
    // rint((x - z) / s) of the rounded quotient: a product with the reciprocal is within 2^-18 of that quotient
    // (both below 32, a few roundings of 2^-24), so only near the middle of two codes is the division made
    const float inv = __frcp_rn(s);
    float near = 0.f, q[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float t = __fmul_rn(__fsub_rn(x[i], z), inv);
      q[i] = rintf(t);
      near = fmaxf(near, fabsf(t - q[i]));
    }
    // also where the reciprocal leaves the range, or x is not a number: then t - q is not one, or not small
    if (!(near < 0.5f - 0x1p-17f) || !(fabsf(inv) < 0x1p120f) || !(fabsf(s) < 0x1p120f)) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = rintf(__fdiv_rn(__fsub_rn(x[i], z), s));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) codes |= (uint32_t)fminf(fmaxf(q[i], 0.0f), 15.0f) << (4 * i);
  }
  return codes;
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t* row, int lane, uint32_t codes) {
  if (N == 2) row[lane] = (uint8_t)codes;
  if (N == 4) reinterpret_cast<uint16_t*>(row)[lane] = (uint16_t)codes;
  if (N == 8) reinterpret_cast<uint32_t*>(row)[lane] = codes;
}

enum { kNeighbours, kLanes, kAnywhere };  // where a column's partner is: beside it, in one other lane, in the row

// The rotation of one lane's columns of any row of a token: x[i] becomes x[i] * cs[i] + partner * sn[i].
template <typename T, int N>
struct Turn {
  float cs[N], sn[N];
  int partner;  // lane of the partner's columns (kLanes)
  int columns;  // how many of this lane's columns rotate
  int mode, n_freq;

  __device__ __forceinline__ Turn(const float2* table, int freqs, bool interleaved, int lane) {
    n_freq = freqs;
    const int apart = freqs / N;
    mode = interleaved ? kNeighbours : freqs % N == 0 ? kLanes : kAnywhere;
    partner = (lane < apart ? lane + apart : lane - apart) & 31;
    columns = max(0, min(N, 2 * freqs - lane * N));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int col = lane * N + i;
      const bool low = interleaved ? !(col & 1) : col < freqs;
      float2 w = make_float2(1.f, 0.f);
      if (i < columns) w = table[interleaved ? col >> 1 : low ? col : col - freqs];
      cs[i] = w.x;
      sn[i] = low ? -w.y : w.y;
    }
  }
  __device__ __forceinline__ void apply(float (&x)[N], const T* row, int lane) const {
    float other[N];
    if (mode == kNeighbours) {
#pragma unroll
      for (int i = 0; i < N; ++i) other[i] = x[i ^ 1];
    } else if (mode == kLanes) {
#pragma unroll
      for (int i = 0; i < N; ++i) other[i] = __shfl_sync(0xffffffffu, x[i], partner);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int col = lane * N + i;
        other[i] = i < columns ? to_f32(row[col < n_freq ? col + n_freq : col - n_freq]) : 0.f;
      }
      __syncwarp();  // the row may be overwritten next: every lane has read its partners
    }
    if (columns == N) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(other[i], sn[i]));
    } else if (columns > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < columns) x[i] = __fadd_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(other[i], sn[i]));
    }
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) * D > 512 ? 2 : 4) kv_append(const fmoe_kv_cache c, const fmoe_kv_tokens a,
                                                                                int parts, int* err) {
  constexpr int N = D / 32, U = 2;  // rows in flight
  __shared__ float2 tables[kWarps][D / 2];                             // cosine, sine
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  const int t = (int)(item / parts), part = (int)(item - (int64_t)t * parts);
  if (t >= a.n_tokens) return;
  const int pos = a.positions[t];
  if (pos < 0) return;
  const T* src = static_cast<const T*>(a.q.ptr) + t * a.q.token_stride + part * a.q.head_stride + lane * N;
  T* dst = static_cast<T*>(a.q_out.ptr) + t * a.q_out.token_stride + part * a.q_out.head_stride + lane * N;
  const int64_t from = parts * a.q.head_stride, into = parts * a.q_out.head_stride;
  Pack<T, N> row[U];
  auto fetch = [&](int r) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u * parts < a.heads_q) row[u] = *reinterpret_cast<const Pack<T, N>*>(src + u * from);
  };
  fetch(part);
  float2* const table = tables[warp];
  for (int i = lane; i < a.n_freq; i += 32) {
    double sn, cs;
    sincos((double)pos * (double)a.inv_freq[i], &sn, &cs);
    table[i] = make_float2((float)cs, (float)sn);
  }
  __syncwarp();
  const Turn<T, N> turn(table, a.n_freq, a.interleaved, lane);
  // ---- query rows
  for (int r = part; r < a.heads_q; r += U * parts) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u * parts < a.heads_q) {
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = to_f32(row[u].v[i]);
        turn.apply(x, src + u * from - lane * N, lane);
        store_f32<T, N>(dst + u * into, x);
      }
    src += U * from;
    dst += U * into;
    fetch(r + U * parts);
  }
  // ---- key and value rows: the warps go on where the query rows ended
  const int first = ((part - a.heads_q) % parts + parts) % parts, ps = c.page_size;
  if (first >= 2 * c.heads) return;
  const size_t block = (size_t)ps * (D + D / 8);
  const Place to = place_of(c, a.positions, a.seq, t, block, err, lane == 0);
  if (!to.block) return;
  for (int r = first; r < 2 * c.heads; r += parts) {
    const int v = r >= c.heads, h = r - v * c.heads;
    const fmoe_view& in = v ? a.v : a.k;
    const T* const at = static_cast<const T*>(in.ptr) + t * in.token_stride + h * in.head_stride;
    float x[N];
    load_f32<T, N>(at + lane * N, x);
    if (!v) turn.apply(x, at, lane);
    uint32_t sb;
    const uint32_t codes = quantise<N>(x, &sb);
    uint8_t* const blk = to.block + h * block;
    store_codes<N>(blk + ((size_t)v * ps + to.at) * (D / 2), lane, codes);
    if (lane % (64 / N) == 0)
      reinterpret_cast<uint32_t*>(blk + (size_t)ps * D)[((size_t)v * ps + to.at) * (D / 64) + lane / (64 / N)] = sb;
  }
}

// A warp reads one row.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv_read(const fmoe_kv_cache c, const int32_t* positions, const int32_t* seq,
                                                    int n_tokens, const fmoe_out_view k, const fmoe_out_view v, int* err) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31, ps = c.page_size;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(item / (2 * c.heads)), r = (int)(item - (int64_t)t * (2 * c.heads));
  if (t >= n_tokens) return;
  const size_t block = (size_t)ps * (D + D / 8);
  const Place at = place_of(c, positions, seq, t, block, err, lane == 0);
  if (!at.block) return;
  const int kind = r >= c.heads, h = r - kind * c.heads;
  const uint8_t* const blk = at.block + h * block;
  const uint8_t* const row = blk + ((size_t)kind * ps + at.at) * (D / 2);
  const uint32_t codes = N == 2   ? row[lane]
                         : N == 4 ? reinterpret_cast<const uint16_t*>(row)[lane]
                                  : reinterpret_cast<const uint32_t*>(row)[lane];
  const uint32_t sb =
      reinterpret_cast<const uint32_t*>(blk + (size_t)ps * D)[((size_t)kind * ps + at.at) * (D / 64) + lane / (64 / N)];
  const float s = __uint_as_float(sb << 16), z = __uint_as_float(sb & 0xffff0000u);
  float x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = fmaf((float)((codes >> (4 * i)) & 15u), s, z);
  const fmoe_out_view& to = kind ? v : k;
  store_f32<T, N>(static_cast<T*>(to.ptr) + t * to.token_stride + h * to.head_stride + lane * N, x);
}

}  // namespace

cudaError_t launch_kv_append(const fmoe_kv_cache& c, const fmoe_kv_tokens& t, int sms, int* err, cudaStream_t st) {
  // all rows of a token a warp, fewer where that leaves the SMs unfilled: its angles are computed once (8192 tokens
  // of 36 rows of 256: 86 us, 206 us with a warp a row; 32 tokens of 40 rows of 128: 17 us, 6.6 us with a warp a row)
  const long long rows = (long long)t.heads_q + 2ll * c.heads;
  const long long parts = std::max(1ll, std::min(rows, 48ll * sms / t.n_tokens));
  const long long blocks = (t.n_tokens * parts + kWarps - 1) / kWarps;
  return with_dtype(t.dtype, [&](auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    const auto kernel = c.dim == 64 ? kv_append<T, 64> : c.dim == 128 ? kv_append<T, 128> : kv_append<T, 256>;
    kernel<<<(unsigned)blocks, kThreads, 0, st>>>(c, t, (int)parts, err);
    return cudaGetLastError();
  });
}

cudaError_t launch_kv_read(const fmoe_kv_cache& c, const int32_t* positions, const int32_t* seq, int n_tokens,
                           int dtype, const fmoe_out_view& k, const fmoe_out_view& v, int* err, cudaStream_t st) {
  const long long blocks = ((long long)n_tokens * 2 * c.heads + kWarps - 1) / kWarps;
  return with_dtype(dtype, [&](auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    const auto kernel = c.dim == 64 ? kv_read<T, 64> : c.dim == 128 ? kv_read<T, 128> : kv_read<T, 256>;
    kernel<<<(unsigned)blocks, kThreads, 0, st>>>(c, positions, seq, n_tokens, k, v, err);
    return cudaGetLastError();
  });
}

}  // namespace fmoe
