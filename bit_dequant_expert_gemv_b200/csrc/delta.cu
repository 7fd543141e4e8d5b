// delta.cu — the gated delta rule, recurrent form (one token after another, binary32 throughout).
//
// A CTA of 128 threads owns 32 columns of one head's state: the columns of a state never mix
// (S'^T k and S^T q are taken column by column), so 32 columns of dim_k rows sit in registers,
// 16 row groups x 8 threads of 4 columns, and every token needs one pass over them. With
// p = S^T k, o = S^T q of the state BEFORE the token and the scalars k.k, q.q, k.q, all five
// reduced together, the rest follows without a second reduction:
//   u = beta (v - e^g kappa p),   out = scale rho (e^g o + kappa (k.q) u),   S = e^g S + kappa k u^T
// with kappa, rho the norms' reciprocals. One barrier per token; the reductions' buffers alternate.
//
// A decode step reads and writes every state once (8 bytes an entry for about 6 flops): it is bound
// by HBM. 32 columns keep 128-byte row segments and give one sequence of 64 heads 256 CTAs. Measured, 64 heads of
// 128 x 128, bf16: 128 requests 175 to 187 us, 94 to 88 % of the copy rate, by the machine; one request 4.1 us, a launch
// with slot, state and sums one after another in it.
#include "api.h"
#include "mixer.h"

namespace fmoe {
namespace {

constexpr int kCols = 32;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// ONE: every sequence is one token (a decode step): nothing is fetched ahead, and more CTAs fit an SM (128 requests
// 175 us, 239 us by the form for several tokens).
template <typename T, int DK, bool ONE>
__global__ void __launch_bounds__(kThreads) delta_recurrent(const DeltaRun r) {
  constexpr int R = DK / 16;  // rows of a thread
  __shared__ float4 red[2][kWarps][8][2];
  __shared__ float dots[2][kWarps][4];
  const fmoe_delta_desc& d = r.d;
  const int slices = d.dim_v / kCols;
  const int i = blockIdx.x / slices, c0 = (blockIdx.x - i * slices) * kCols, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = c0 + 4 * (lane & 7), row = (warp * 4 + (lane >> 3)) * R;

  int64_t t = i, end = i + 1;
  if (!ONE) {
    t = r.cu[i];
    end = r.cu[i + 1];
    if (t < 0 || end < t || end > r.n_tokens) {
      if (threadIdx.x == 0) report(r.err, ERR_LENGTH);
      return;
    }
    if (t == end) return;
  }
  const int slot = d.slots ? d.slots[i] : i;
  if (slot < 0 || slot >= d.n_slots) {
    if (threadIdx.x == 0 && slot >= 0) report(r.err, ERR_SLOT);
    return;
  }
  float* const state = d.state + slot * d.state_stride + ((int64_t)h * DK + row) * d.dim_v + col;
  float4 s[R];
  if (r.fresh && r.fresh[i]) {
#pragma unroll
    for (int j = 0; j < R; ++j) s[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
#pragma unroll
    for (int j = 0; j < R; ++j) s[j] = *reinterpret_cast<const float4*>(state + (int64_t)j * d.dim_v);
  }
  const int hk = h / (d.heads_v / d.heads_k);
  const T* const q = static_cast<const T*>(d.q.ptr) + hk * d.q.head_stride + row;
  const T* const k = static_cast<const T*>(d.k.ptr) + hk * d.k.head_stride + row;
  const T* const v = static_cast<const T*>(d.v.ptr) + h * d.v.head_stride + col;
  T* const out = static_cast<T*>(d.out.ptr) + h * d.out.head_stride + col;

  float kn[R], qn[R], vn[4], gn, bn;  // the next token's
  auto fetch = [&](int64_t at) {
    load_f32<T, R>(k + at * d.k.token_stride, kn);
    load_f32<T, R>(q + at * d.q.token_stride, qn);
    load_f32<T, 4>(v + at * d.v.token_stride, vn);
    gn = d.g[at * d.gate_stride + h];
    bn = d.beta[at * d.gate_stride + h];
  };
  fetch(t);
  for (int buf = 0; t < end; ++t, buf ^= 1) {
    float kc[R], qc[R], vc[4];
    const float g = gn, beta = bn;
#pragma unroll
    for (int j = 0; j < R; ++j) kc[j] = kn[j], qc[j] = qn[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) vc[j] = vn[j];
    if (!ONE && t + 1 < end) fetch(t + 1);
    float x[11] = {};  // p (4), o (4), k.k, q.q, k.q
#pragma unroll
    for (int j = 0; j < R; ++j) {
      x[0] = fmaf(s[j].x, kc[j], x[0]);
      x[1] = fmaf(s[j].y, kc[j], x[1]);
      x[2] = fmaf(s[j].z, kc[j], x[2]);
      x[3] = fmaf(s[j].w, kc[j], x[3]);
      x[4] = fmaf(s[j].x, qc[j], x[4]);
      x[5] = fmaf(s[j].y, qc[j], x[5]);
      x[6] = fmaf(s[j].z, qc[j], x[6]);
      x[7] = fmaf(s[j].w, qc[j], x[7]);
      x[8] = fmaf(kc[j], kc[j], x[8]);
      x[9] = fmaf(qc[j], qc[j], x[9]);
      x[10] = fmaf(kc[j], qc[j], x[10]);
    }
#pragma unroll
    for (int m = 8; m < 32; m <<= 1)
#pragma unroll
      for (int j = 0; j < 11; ++j) x[j] += __shfl_xor_sync(0xffffffffu, x[j], m);
    if (lane < 8) {
      red[buf][warp][lane][0] = make_float4(x[0], x[1], x[2], x[3]);
      red[buf][warp][lane][1] = make_float4(x[4], x[5], x[6], x[7]);
      if (lane == 0) {
        dots[buf][warp][0] = x[8];
        dots[buf][warp][1] = x[9];
        dots[buf][warp][2] = x[10];
      }
    }
    __syncthreads();
    float p[4] = {}, o[4] = {}, kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 a = red[buf][w][lane & 7][0], b = red[buf][w][lane & 7][1];
      p[0] += a.x, p[1] += a.y, p[2] += a.z, p[3] += a.w;
      o[0] += b.x, o[1] += b.y, o[2] += b.z, o[3] += b.w;
      kk += dots[buf][w][0];
      qq += dots[buf][w][1];
      kq += dots[buf][w][2];
    }
    const float eg = expf(g);
    // a row of zeros stays one where eps is zero too (a NaN takes the first branch)
    const float kappa = d.l2norm ? (kk + d.eps != 0.f ? 1.0f / sqrtf(kk + d.eps) : 0.f) : 1.0f;
    const float rho = d.scale * (d.l2norm ? (qq + d.eps != 0.f ? 1.0f / sqrtf(qq + d.eps) : 0.f) : 1.0f);
    const float decay = eg * kappa, own = kappa * kq;
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = beta * (vc[j] - decay * p[j]);
      o[j] = rho * (eg * o[j] + own * u[j]);
    }
    if (row == 0) store_f32<T, 4>(out + t * d.out.token_stride, o);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float kj = kappa * kc[j];
      s[j].x = fmaf(kj, u[0], eg * s[j].x);
      s[j].y = fmaf(kj, u[1], eg * s[j].y);
      s[j].z = fmaf(kj, u[2], eg * s[j].z);
      s[j].w = fmaf(kj, u[3], eg * s[j].w);
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) *reinterpret_cast<float4*>(state + (int64_t)j * d.dim_v) = s[j];
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaRun& r, cudaStream_t st) {
  const dim3 grid((unsigned)r.n * (unsigned)(r.d.dim_v / kCols), (unsigned)r.d.heads_v);
  return with_dtype(r.d.dtype, [&](auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    const auto kernel = r.d.dim_k == 64 ? (r.cu ? delta_recurrent<T, 64, false> : delta_recurrent<T, 64, true>)
                                        : (r.cu ? delta_recurrent<T, 128, false> : delta_recurrent<T, 128, true>);
    kernel<<<grid, kThreads, 0, st>>>(r);
    return cudaGetLastError();
  });
}

}  // namespace fmoe
