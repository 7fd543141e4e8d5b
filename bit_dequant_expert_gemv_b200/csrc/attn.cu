// attn.cu — attention over the paged 4-bit cache.
//
// Per query row: out = sum_t p_t v_hat_t, p = softmax_t(scale q . k_hat_t), x_hat = code * s + z for
// every 64 columns. The scales stay out of the matrix products:
//   q . k_hat_t     = sum over groups of  s_t (q . code_t) + z_t (sum of q)
//   sum_t p_t v_hat = sum over groups of  sum_t (p_t s_t) code_t + sum_t p_t z_t
// so that both products multiply the codes themselves. A code's four bits, masked in place, ARE a
// binary16 number: code * 2^-24 (bits 0..3) or code * 2^-20 (bits 4..7), both subnormal and exact, so
// unpacking is one AND per two codes and one shift per eight; the powers of two go into q and out. (For binary16 and
// binary32 results one more instruction makes them normal numbers.)
//
// One warp takes 16 positions at a time, as the ROWS of m16n8k16 products, 8 query rows as the
// columns: the heads that share a kv head fill a tile without waste at 8, and the scores come out
// in the registers that the second product (value columns x positions times positions x query rows)
// wants transposed, one movmatrix each. The order of columns inside a product is free, so that a
// thread takes whole words of codes into its fragments: for keys two words of a group, for values the
// words of the two positions of a pair, spliced by byte permutes.
//
// Every warp (or every group of warps on different rows of the same positions) streams its own
// positions, 32 at a time, through a ring of stages filled by asynchronous copies: the loads in flight
// cost no registers, and no barrier joins the CTA before the end. 16-byte chunks of a stage are
// permuted so that the reads above meet no bank conflict.
//
// Work is cut in passes of 32 positions per warp. All passes of all (sequence, kv head, block of rows)
// items stand in one row, and every CTA takes an equal share of it, wherever items begin and end:
// lengths of any mixture keep every SM busy to the end. (Of sequences with like numbers of queries: every sequence
// counts the blocks of rows that max_q gives, and the CTAs that get empty ones are done at once. A long prompt among
// single queries runs on the few CTAs that its share of the positions gives it.) What a CTA has of an item that others
// share goes to scratch (at most its first and its last item), and a second launch joins the parts, in order.
//
// Measured, 32 query heads: 32 requests of up to 8192 positions, 4 kv heads of 128: 44 us for bfloat16, 53 for binary16,
// 58 for binary32; one of 262144, 2 of 256: 73, 97 and 119 us, of which 23 us would be the codes' bytes at the copy
// rate. Instructions bound it, and that each waits for the one before: unpacking, scales and softmax take 29.9 million
// warp instructions for the long one in bfloat16, issued in 44 % of the cycles by the two warps of a scheduler whose
// registers the sums leave room for (54 % by the four warps at 128 columns). At 256 columns and 16 rows 255 registers
// do not hold them all: 240 bytes are stored and 252 loaded again. One request of 777 positions: 14 us, seven stages of
// 32 one after another.
#include "api.h"
#include "mixer.h"
#include "mma.cuh"
#include "ptx.cuh"

namespace fmoe {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnRun {
  fmoe_kv_cache c;
  fmoe_attn_desc a;
  AttnPlan p;
  float* part;   // [CTAs][2][rows of a CTA][dim]
  float2* stat;  // [CTAs][2][rows of a CTA]: maximum (base-2 logits), sum
  int* err;
};

// The queries and the length of sequence i, checked: q0, number of queries, positions in the cache.
struct Seq {
  int q0, nq, len;
  int limit;  // positions that may be read
};
__device__ __forceinline__ Seq seq_of(const AttnRun& r, int i, bool tell) {
  Seq s;
  s.q0 = r.a.cu_q ? r.a.cu_q[i] : i;
  const int q1 = r.a.cu_q ? r.a.cu_q[i + 1] : i + 1;
  s.len = r.a.lens[i];
  const bool queries = s.q0 >= 0 && q1 >= s.q0 && q1 <= r.a.n_tokens;  // compared, not subtracted: any numbers may stand there
  s.nq = queries ? q1 - s.q0 : 0;
  const long long room = (long long)r.c.max_pages * r.c.page_size;
  s.limit = (int)min((long long)min(max(s.len, 0), r.a.max_len), room);
  if (tell && (!queries || s.len != s.limit || s.nq > r.a.max_q)) report(r.err, ERR_LENGTH);
  return s;
}
// Positions seen by query j of a sequence.
__device__ __forceinline__ int seen(const Seq& s, int j) {
  return (int)min((long long)s.limit, max(0ll, (long long)s.len - s.nq + j + 1));
}

constexpr int kStage = 32;  // positions of a stage, and of a pass
constexpr int kStages = 2;  // of a ring: three gained nothing at any of the sizes below

// Passes of a sequence: none without queries, else at least one (a query that sees nothing gives zeros).
__device__ __forceinline__ int passes_of(const AttnRun& r, int i) {
  if (r.a.cu_q && r.a.cu_q[i + 1] <= r.a.cu_q[i]) return 0;
  const long long room = (long long)r.c.max_pages * r.c.page_size;
  const int len = (int)min((long long)min(max(r.a.lens[i], 0), r.a.max_len), room);
  return max(1, (len + kStage - 1) / kStage);
}

// A place in the row of all passes: pass `pass` of `n` of item `unit` (kv head and block of rows) of
// sequence i. Every lane of a warp holds the same.
struct Place {
  int i, unit, pass, n;
};
// The passes of the sequences, for one unit: all of them, and (where asked for) those before `until`.
__device__ __forceinline__ long long total_passes(const AttnRun& r, int lane, int until = 0, long long* before = nullptr) {
  long long sum = 0, first = 0;
  for (int i = lane; i < r.c.n_seqs; i += 32) {
    const int n = passes_of(r, i);
    sum += n;
    if (i < until) first += n;
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (before) first += __shfl_xor_sync(0xffffffffu, first, m);
  }
  if (before) *before = first;
  return sum;
}
// The place of pass `at` (below the total) of the whole row: sequence by sequence, in each unit by unit.
__device__ __forceinline__ Place find_pass(const AttnRun& r, long long at, int units, int lane) {
  for (int base = 0; base < r.c.n_seqs; base += 32) {
    const int n = base + lane < r.c.n_seqs ? passes_of(r, base + lane) : 0;
    long long sum = (long long)n * units;  // inclusive
    for (int m = 1; m < 32; m <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, sum, m);
      if (lane >= m) sum += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, sum > at);
    if (past) {
      const int l = __ffs(past) - 1, nl = __shfl_sync(0xffffffffu, n, l);
      const long long in = at - (__shfl_sync(0xffffffffu, sum, l) - (long long)nl * units);  // may pass 2^31
      return {base + l, (int)(in / nl), (int)(in % nl), nl};
    }
    at -= __shfl_sync(0xffffffffu, sum, 31);
  }
  return {r.c.n_seqs, 0, 0, 0};
}
// The CTAs that share all passes: no more than there are passes, so that each has one (the host knows only a
// bound of the lengths), and every part of a cut item is written.
__device__ __forceinline__ int sharers(const AttnRun& r, long long total) { return (int)min((long long)r.p.ctas, total); }
// The first pass of CTA b of `of`.
__device__ __forceinline__ long long share_begin(long long total, int b, int of) {
  return total / of * b + (total % of) * b / of;
}

// A stage: key codes [32][dim/2 bytes], value codes, key sb [32][NG words], value sb. Row `r` of a 16-row
// piece of codes has 2 NG chunks of 16 bytes; chunk q lies at slot (row's first slot + q) ^ mask(r).
// A key read takes one 32-byte group of rows 0, 4, 1, 5 (then 2, 6, 3, 7) at once, a value read of rows
// 4j .. 4j+3: the masks give the four rows different pairs of the eight 16-byte slots of the banks.
template <int NG>
struct Stage {
  static constexpr int kRow = NG * 32;  // bytes of a row of codes
  static constexpr int kV = kStage * kRow, kKs = 2 * kV, kVs = kKs + kStage * NG * 4;
  static constexpr int kBytes = kVs + kStage * NG * 4;
  static __device__ __forceinline__ int key_mask(int r) {
    return NG == 1 ? 4 * ((r >> 2) & 1) : NG == 2 ? 2 * ((r >> 2) & 1) : 2 * ((r & 1) | ((r >> 1) & 2));
  }
  static __device__ __forceinline__ int value_mask(int r) {
    return NG == 1 ? 4 * ((r >> 2) & 1) : NG == 2 ? 2 * ((r >> 1) & 1) : 2 * (r & 3);
  }
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[0] = a.x, w[1] = a.y;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
}

__device__ __forceinline__ float scale_of(uint32_t sb) { return __uint_as_float(sb << 16); }
__device__ __forceinline__ float bias_of(uint32_t sb) { return __uint_as_float(sb & 0xffff0000u); }

// p s / 2^E is held in binary16 times 2^kLift. The running maximum follows the scores' only when they pass it
// by kSlack (base 2), and E is set one above a scale's exponent: most stages then leave the sums as they are. A
// scale is below 2^(E + 1), so p s stays below 2^(kLift + kSlack + 1) = 2^15, and it is a normal number down to
// 2^-22 of 2^E; below that it is held to 2^-33 of 2^E, 2^-32 of the largest scale. The exponent goes by the scales and not by
// p s: that would take another maximum of every row, three shuffles a row and stage.
constexpr int kLift = 8, kSlack = 6;
constexpr int kMinE = kLift;
// Stages of a ring that are not worth sharing (1024 positions). An item whole and shared, us: 4 items of 256, 777 and 1024
// positions 8.5 and 11.6, 14.4 and 15.8, 15.7 and 16.4; 128 items 8.9 and 20.5, 13.7 and 23.1, 15.7 and 23.4. One item
// alone (a request with one kv head) is better shared from 777 positions on: 14.3 and 11.2, 15.7 and 11.6.
constexpr int kShort = 8;

// How the operands of the two products are held for results of type T, beside sums of binary32.
//   q: binary16 parts of a query. One holds a 16-bit query as it is, two a binary32 one (22 bits).
//   ps: binary16 parts of p s. One (2^-12) is far below a bfloat16 result's own rounding of 2^-8. A binary16 result's is
//     2^-11: one part more than doubled its error, as p s multiplies codes of mean 7.5 that the biases take back out (64
//     to 20000 positions of like weight: 4.3e-4 to 4.9e-4 in one part, 2.0e-4 to 2.2e-4 in two, which is the rounding
//     of the result; 12 requests of 5 queries, 64 columns: 37 us in one part, 41 us in two; the long request of the
//     file's head 72 and 97 us).
//   normal: codes as normal numbers. Sums of products drop what lies below 2^-24 of the largest exponent among them, and
//     a subnormal counts there as 2^10 times what it is: with codes in place a binary32 result was up to 4e-5 off.
template <typename T>
struct Held {
  static constexpr int q = sizeof(T) == 4 ? 2 : 1, ps = std::is_same<T, __nv_bfloat16>::value ? 1 : 2;
  static constexpr bool normal = ps == 2;
};
int terms_of(int dtype) { return dtype == FMOE_F32 ? 2 : 1; }  // Held::q

// CTAs of an SM, by the registers that their sums take.
__host__ __device__ constexpr int resident(int ng, int nt, int terms) {
  return ng * nt * terms <= 2 ? 4 : ng * nt * terms <= 3 ? 3 : 2;
}
// Tiles of 8 rows that a warp can carry.
__host__ __device__ constexpr int most_tiles(int ng) { return ng == 1 ? 4 : ng == 2 ? 3 : 2; }

// Two codes as they go into a product, less `middle` where they are normal numbers: x_hat = (code - 8) s + (z + 8 s), so
// that the sums of values are of about the results' size and not of the codes' (131072 positions of like weight, 14000 of
// them in a row: binary32 results 9.8e-5 off without it).
constexpr int kMiddle = 8;
template <bool NORMAL>
__device__ __forceinline__ uint32_t codes_in(uint32_t masked, int middle = 0) {
  if (!NORMAL) return masked;
  uint32_t d;
  const uint32_t base = 0x6400u + middle;  // 1024 + code - (1024 + middle), exact
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(masked | 0x64006400u), "r"(base << 16 | base));
  return d;
}
template <typename T, int NG, int NT>
__global__ void __launch_bounds__(kThreads, resident(NG, NT, Held<T>::q)) attn_kernel(const AttnRun r) {
  constexpr int TERMS = Held<T>::q, PS = Held<T>::ps;
  constexpr bool NORMAL = Held<T>::normal;
  constexpr int D = NG * 64, MT = NG * 4;
  constexpr int ROWS = 8 * NT;  // of a warp
  using L = Stage<NG>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 wstat[kWarps][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int group = r.a.heads_q / r.c.heads, units = r.c.heads * r.p.row_blocks;
  const int rw = warp % r.p.row_warps, tw = warp / r.p.row_warps, tws = kWarps / r.p.row_warps;
  const int step = kStage * tws, ps = r.c.page_size;
  const size_t block_bytes = (size_t)ps * (D + D / 8), page_bytes = r.c.heads * block_bytes;
  const uint32_t my_ring = smem_u32(ring) + tw * kStages * L::kBytes;
  // this lane's slots in a piece's rows of keys and of values, and the distances between its chunks in a block
  const uint32_t key_slot = (lane ^ L::key_mask(lane / (2 * NG))) * 16;
  const uint32_t value_slot = L::kV + (lane ^ L::value_mask(lane / (2 * NG))) * 16;
  const int half = ps * L::kRow, sb_half = ps * NG * 4;
  // the quarters of a stage (piece, half) that this warp copies for its ring
  const uint32_t quarters = r.p.row_warps == 1 ? 15u : r.p.row_warps == 2 ? 3u << (2 * rw) : 1u << rw;
  uint4* const q_frag = reinterpret_cast<uint4*>(ring + r.p.q_offset);                       // [warp rows][n][y][term][2][lane]
  float* const q_stat = reinterpret_cast<float*>(q_frag + r.p.row_warps * (NT * NG * TERMS * 64));  // [row][NG + 1]
  // positions c, c+4, c+8, c+12 of a piece are the columns 2c, 2c+1, 2c+8, 2c+9 of the value product
  const int tok = (g >> 1) + 4 * (g & 1);  // and so this and + 8 the rows g, g+8 of the scores
  const int key_at = tok * L::kRow + 8 * (c & 1) + 16 * (c >> 1), key_mask = 16 * L::key_mask(tok);
  // a word of a value row c + 4j: NG = 1 masks 4 (j & 1), the others by c
  auto value_at = [&](int y, int j) {
    return NG == 1 ? (c * L::kRow + 4 * g) ^ (64 * (j & 1)) : (c * L::kRow + 4 * g + 32 * y) ^ (16 * L::value_mask(c));
  };

  cudaTriggerProgrammaticLaunchCompletion();  // the joining launch may be set up; it waits for this one's end
  // Counts and lengths out of range, of sequences without queries too: an item's first CTA, or the first of all.
  if (r.p.by_item) {
    if (blockIdx.x % units == 0 && threadIdx.x == 0) seq_of(r, blockIdx.x / units, true);
  } else if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < r.c.n_seqs; i += kThreads) seq_of(r, i, true);
  }
  long long now, last;
  Place at;
  if (r.p.by_item) {
    at = {(int)(blockIdx.x / units), (int)(blockIdx.x % units), 0, 0};
    at.n = passes_of(r, at.i);
    now = 0, last = at.n;
  } else {
    const long long total = total_passes(r, lane) * units;
    const int of = sharers(r, total);
    if ((int)blockIdx.x >= of) return;
    last = share_begin(total, blockIdx.x + 1, of);
    now = share_begin(total, blockIdx.x, of);
    at = find_pass(r, now, units, lane);
  }
  if (now >= last) return;
  for (;;) {
  const int i = at.i, h = at.unit / r.p.row_blocks, rb = at.unit - h * r.p.row_blocks;
  const int passes = (int)min((long long)(at.n - at.pass), last - now);  // of this item
  const Seq s = seq_of(r, i, false);
  const int block_row = rb * r.p.row_warps * ROWS, rows = min(s.nq, r.a.max_q) * group;
  if (block_row < rows) {
  const int block_seen = seen(s, min(rows - 1, block_row + r.p.row_warps * ROWS - 1) / group);
  const int begin = at.pass * kStage, end = min(begin + passes * kStage, block_seen);

  // ---- positions of this warp: stages of 32 from begin + 32 tw on, every tws-th. A lane looks up the page of
  // one of the next 32 pieces.
  const uint8_t* const pages = static_cast<const uint8_t*>(r.c.pages) + h * block_bytes + lane * 16;
  const int32_t* const table = r.c.page_table + i * r.c.table_stride;
  const int first = begin + kStage * tw;
  const int n_it = first < end ? (end - first + step - 1) / step : 0;
  int off = -1, fetch_slot = 0;  // a lane's piece: its place in its page (-1: there is none)
  uint32_t from_lo = 0, from_hi = 0;  // and the distance of its first key row from `pages`
  uint32_t flags = 0;  // two bits a stage: which pieces are there
  auto sync_ring = [&]() {
    if (r.p.row_warps == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + tw), "r"(32 * r.p.row_warps) : "memory");
  };
  auto fetch = [&](int it) {
    if (it < n_it) {
      if ((it & 15) == 0) {
        const int pos = first + (it + (lane >> 1)) * step + 16 * (lane & 1);
        off = -1;
        if (pos < end) {
          const int j = pos / ps, page = __ldg(table + j);
          if (page >= 0 && page < r.c.n_pages) {
            off = pos - j * ps;
            const size_t from = page * page_bytes + off * L::kRow;
            from_lo = (uint32_t)from;
            from_hi = (uint32_t)(from >> 32);
          } else {
            report(r.err, ERR_PAGE);
          }
        }
      }
      uint32_t to = my_ring + fetch_slot * L::kBytes, ok = 0;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int at = __shfl_sync(0xffffffffu, off, (2 * it + p) & 31);
        const uint32_t lo = __shfl_sync(0xffffffffu, from_lo, (2 * it + p) & 31);
        const uint32_t hi = __shfl_sync(0xffffffffu, from_hi, (2 * it + p) & 31);
        if (at < 0) continue;
        ok |= 1u << p;
        const uint8_t* const k = pages + ((size_t)hi << 32 | lo);
        const uint8_t* const sb = k + (2 * half - at * (L::kRow - NG * 4));
        // 32 chunks on, a row's mask is the same, but for keys of four groups: 4 rows on
        if (quarters >> (2 * p) & 1) {
#pragma unroll
          for (int j = 0; j < NG; ++j)
            copy16(to + p * 16 * L::kRow + 512 * j + (NG == 4 ? key_slot ^ (64 * (j & 1)) : key_slot), k + 512 * j);
          if (lane < 4 * NG) copy16(to + L::kKs + p * 64 * NG + lane * 16, sb);
        }
        if (quarters >> (2 * p) & 2) {
#pragma unroll
          for (int j = 0; j < NG; ++j) copy16(to + p * 16 * L::kRow + 512 * j + value_slot, k + half + 512 * j);
          if (lane < 4 * NG) copy16(to + L::kVs + p * 64 * NG + lane * 16, sb + sb_half);
        }
      }
      flags = (flags & ~(3u << (2 * fetch_slot))) | ok << (2 * fetch_slot);
    }
    copy_commit();
    fetch_slot ^= 1;
  };
  fetch(0);

  // ---- queries, as fragments: a thread takes one word's columns (8) of one row
  for (int k = threadIdx.x; k < r.p.row_warps * ROWS * (D / 8); k += kThreads) {
    const int rr = k / (D / 8), w = k - rr * (D / 8), row = block_row + rr;
    float q[8] = {};
    if (row < rows)
      load_f32<T, 8>(static_cast<const T*>(r.a.q.ptr) + (s.q0 + row / group) * r.a.q.token_stride +
                         (h * group + row % group) * r.a.q.head_stride + 8 * w, q);
    float mx = 0.f, sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(q[j]));
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    // the row's largest value brought to [2^10, 2^11): products with code * 2^-24 stay far inside binary32
    const int e = max(-115, min(103, exponent(mx))) - 10;
    const float f = r.a.scale < 0.f ? -pow2i(-e) : pow2i(-e);  // logits grow with the products
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q[j] *= f;
      sum += q[j];
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if ((w & 7) == 0) q_stat[rr * (NG + 1) + (w >> 3)] = sum * (NORMAL ? 1.0f : 5.9604644775390625e-8f);  // as the codes: 2^-24
    if (w == 0) q_stat[rr * (NG + 1) + NG] = fmaxf(pow2i(e) * fabsf(r.a.scale) * (NORMAL ? kLog2e : kLog2e * 16777216.0f), 1e-37f);
    // codes j, j+4 of a word share a register; odd ones stand 4 bits higher: 16 times larger
    uint32_t a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = q[j] * ((j & 1) ? 0.0625f : 1.0f), hi = q[j + 4] * ((j & 1) ? 0.0625f : 1.0f);
      a[j] = pack_half2(lo, hi);
      if (TERMS == 2) b[j] = rest_half2(lo, hi, a[j]);
    }
    uint4* const to = q_frag + (((rr >> 3) * NG + (w >> 3)) * TERMS) * 64 + (w & 1) * 32 + (rr & 7) * 4 + ((w & 7) >> 1);
    to[0] = make_uint4(a[0], a[1], a[2], a[3]);
    if (TERMS == 2) to[64] = make_uint4(b[0], b[1], b[2], b[3]);
  }
  __syncthreads();
  const int row0 = block_row + rw * ROWS;
  float lsc[NT][2], qsum[NT][NG][2];
  int vis[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int rr = rw * ROWS + 8 * n + 2 * c + j, row = block_row + rr;
      lsc[n][j] = q_stat[rr * (NG + 1) + NG];
#pragma unroll
      for (int y = 0; y < NG; ++y) qsum[n][y][j] = q_stat[rr * (NG + 1) + y];
      vis[n][j] = row < rows ? seen(s, row / group) : 0;
    }
  const bool worker = row0 < rows;
  const int first_seen = seen(s, block_row / group);  // the least of the CTA's rows; the most is block_seen
  const int last_seen = worker ? seen(s, min(rows - 1, row0 + ROWS - 1) / group) : 0;  // the most of the warp's
  const uint4* const q_mine = q_frag + rw * (NT * NG * TERMS * 64) + lane;

  float o[NT][MT][4] = {}, m[NT][2], l[NT][2] = {}, zs[NT][NG][2] = {};
#pragma unroll
  for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY;
  int E = kMinE;  // biased exponent of the largest value scale so far

  uint8_t* const mine = ring + (size_t)tw * kStages * L::kBytes;
  int slot = 0;
  for (int it = 0; it < n_it; ++it) {
    copy_wait<0>();
    sync_ring();
    fetch(it + 1);
    uint8_t* const st = mine + slot * L::kBytes;
    const uint32_t ok = (flags >> (2 * slot)) & 3u;
    slot ^= 1;
    const int pos = first + it * step;
    const bool tail = ok != 3 || pos + kStage > first_seen;
    if (tail) {
      // Not every row sees every position here. What none sees may hold anything: its scales and biases become
      // zeros. One that only some rows see, if it is not finite, makes those rows' results NaN, and no others'.
      const bool any = pos + lane < block_seen && (ok >> (lane >> 4) & 1u);
      bool odd = false;
      uint32_t* const ks = reinterpret_cast<uint32_t*>(st + L::kKs) + lane * NG;
      uint32_t* const vs = reinterpret_cast<uint32_t*>(st + L::kVs) + lane * NG;
#pragma unroll
      for (int y = 0; y < NG; ++y)
        odd |= ((ks[y] & 0x7f80u) == 0x7f80u) | ((ks[y] & 0x7f800000u) == 0x7f800000u) |
               ((vs[y] & 0x7f80u) == 0x7f80u) | ((vs[y] & 0x7f800000u) == 0x7f800000u);
      const uint32_t odd_seen = __ballot_sync(0xffffffffu, odd && any);
      sync_ring();  // every warp of the ring has looked
      if (!any || odd)
#pragma unroll
        for (int y = 0; y < NG; ++y) ks[y] = vs[y] = 0u;
      sync_ring();
      if (odd_seen)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int k = vis[n][j] - pos;
            if (k > 0 && (odd_seen & (k >= 32 ? ~0u : (1u << k) - 1u))) l[n][j] = NAN;
          }
    }
    if (pos >= last_seen || ok == 0) continue;
    // ---- scores: positions tok, tok+8 of both pieces against rows 2c, 2c+1
    float x[NT][2][4];
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      uint32_t q[NT][TERMS][8];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < TERMS; ++e) {
          const uint4* const from = q_mine + ((n * NG + y) * TERMS + e) * 64;
          const uint4 lo = from[0], hi = from[32];
          q[n][e][0] = lo.x, q[n][e][1] = lo.y, q[n][e][2] = lo.z, q[n][e][3] = lo.w;
          q[n][e][4] = hi.x, q[n][e][5] = hi.y, q[n][e][6] = hi.z, q[n][e][7] = hi.w;
        }
      uint2 k[2][2];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          k[p][j] = *reinterpret_cast<const uint2*>(st + (16 * p + 8 * j) * L::kRow + ((key_at + 32 * y) ^ key_mask));
      float acc[NT][2][4];
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t a = (w ? k[p][0].y : k[p][0].x) >> (8 * u), b = (w ? k[p][1].y : k[p][1].x) >> (8 * u);
            const uint32_t a0 = codes_in<NORMAL>(a & 0x000f000fu), a1 = codes_in<NORMAL>(b & 0x000f000fu);
            const uint32_t a2 = codes_in<NORMAL>(a & 0x00f000f0u), a3 = codes_in<NORMAL>(b & 0x00f000f0u);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < TERMS; ++e)
                if (w + u + e == 0)
                  mma_first(acc[n][p], a0, a1, a2, a3, q[n][e][0], q[n][e][1]);
                else
                  mma(acc[n][p], a0, a1, a2, a3, q[n][e][4 * w + 2 * u], q[n][e][4 * w + 2 * u + 1]);
          }
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t sb = *reinterpret_cast<const uint32_t*>(st + L::kKs + ((16 * p + tok + 8 * j) * NG + y) * 4);
          const float s = scale_of(sb), z = bias_of(sb);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              x[n][p][2 * j + i] = fmaf(acc[n][p][2 * j + i], s,
                                        y ? fmaf(z, qsum[n][y][i], x[n][p][2 * j + i]) : z * qsum[n][y][i]);
        }
    }
    // ---- running maximum of each row, running exponent of the value scales
    uint32_t vs[2][2][NG];
    float ts = 0.f;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        load_words<NG>(st + L::kVs + (16 * p + tok + 8 * j) * NG * 4, vs[p][j]);
#pragma unroll
        for (int y = 0; y < NG; ++y) ts = fmaxf(ts, fabsf(scale_of(vs[p][j][y])));
      }
    int top = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(ts)) >> 23);
    if (top == 255) {  // an infinite scale spoils its own 64 columns; the others keep the exponent of what is finite
      ts = 0.f;
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            const float s = fabsf(scale_of(vs[p][j][y]));
            if (s < INFINITY) ts = fmaxf(ts, s);
          }
      top = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(ts)) >> 23);
    }
    const int En = top > E ? top + 1 : E;
    if (tail) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int k = (ok >> p & 1u) ? vis[n][j] - pos - 16 * p : 0;
            if (tok >= k) x[n][p][j] = -INFINITY;
            if (tok + 8 >= k) x[n][p][j + 2] = -INFINITY;
          }
    }
    float tm[NT][2];
    bool grew = En > E;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float t = fmaxf(fmaxf(x[n][0][j], x[n][0][j + 2]), fmaxf(x[n][1][j], x[n][1][j + 2]));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        tm[n][j] = t * lsc[n][j];
        grew |= tm[n][j] > m[n][j] + kSlack;
      }
    if (__any_sync(0xffffffffu, grew)) {
      const float shrink = En - E > 126 ? 0.f : pow2i(E - En);
      E = En;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float mn = fmaxf(m[n][j], tm[n][j]);
          const float f = mn == -INFINITY ? 1.0f : exp2_fast(m[n][j] - mn);
          m[n][j] = mn;
          l[n][j] *= f;
#pragma unroll
          for (int y = 0; y < NG; ++y) zs[n][y][j] *= f;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            o[n][t][j] *= f * shrink;
            o[n][t][j + 2] *= f * shrink;
          }
        }
    }
    // ---- probabilities, and their products with scales and biases
    const float lift = pow2i(min(127, 127 + kLift - E));
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float ref = m[n][j] == -INFINITY ? 0.f : m[n][j];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float& v = x[n][p][2 * i + j];
            v = exp2_fast(fmaf(v, lsc[n][j], -ref));
            l[n][j] += v;
          }
      }
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      uint32_t b[2][NT][2][PS], a[2][4];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float s0 = scale_of(vs[p][0][y]), z0 = bias_of(vs[p][0][y]), s1 = scale_of(vs[p][1][y]), z1 = bias_of(vs[p][1][y]);
        if (NORMAL) z0 = fmaf(kMiddle, s0, z0), z1 = fmaf(kMiddle, s1, z1);
        s0 *= lift, s1 *= lift;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float* const q = x[n][p];
          const float w0 = q[0] * s0, w1 = q[1] * s0, w2 = q[2] * s1, w3 = q[3] * s1;
          zs[n][y][0] = fmaf(q[0], z0, fmaf(q[2], z1, zs[n][y][0]));
          zs[n][y][1] = fmaf(q[1], z0, fmaf(q[3], z1, zs[n][y][1]));
          const uint32_t lo = pack_half2(w0, w1), hi = pack_half2(w2, w3);
          b[p][n][0][0] = transpose8(lo);
          b[p][n][1][0] = transpose8(hi);
          if (PS == 2) {
            b[p][n][0][PS - 1] = transpose8(rest_half2(w0, w1, lo));
            b[p][n][1][PS - 1] = transpose8(rest_half2(w2, w3, hi));
          }
        }
        // values: rows g (codes 0..3 of a word) and g+8 (codes 4..7), columns the positions
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = *reinterpret_cast<const uint32_t*>(st + L::kV + (16 * p + 4 * j) * L::kRow + value_at(y, j));
        a[p][0] = __byte_perm(v[0], v[1], 0x5410), a[p][1] = __byte_perm(v[0], v[1], 0x7632);
        a[p][2] = __byte_perm(v[2], v[3], 0x5410), a[p][3] = __byte_perm(v[2], v[3], 0x7632);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t m[2][4];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            m[p][j] = codes_in<NORMAL>(a[p][j] & ((t & 1) ? 0x00f000f0u : 0x000f000fu), (t & 1) ? kMiddle * 16 : kMiddle);
            if (t == 1) a[p][j] >>= 8;
          }
        // A stage's products are summed by themselves and added outside, rounded to nearest: the products' own sums drop
        // what does not fit, always to the same side (binary32 results: not even four products are summed so).
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float part[4];
#pragma unroll
          for (int i = 0; i < 2 * PS; ++i) {
            const int p = i / PS, e = i % PS;
            if (i == 0 || TERMS == 2)
              mma_first(part, m[p][0], m[p][1], m[p][2], m[p][3], b[p][n][0][e], b[p][n][1][e]);
            else
              mma(part, m[p][0], m[p][1], m[p][2], m[p][3], b[p][n][0][e], b[p][n][1][e]);
            if (i == 2 * PS - 1 || TERMS == 2)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[n][4 * y + t][j] += part[j];
          }
        }
      }
    }
  }
  copy_wait<0>();
  __syncthreads();

  // ---- this warp's rows into shared memory: sums over positions (lanes of one c), then out = 2^24-fold codes + biases
  float* const smem = reinterpret_cast<float*>(ring);
  float* const to_rows = smem + warp * ROWS * D;
  const float f = pow2i(min(E, 254) - 127), up = (NORMAL ? 1.0f : 16777216.0f) / (1 << kLift);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float sum = l[n][j];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (g == 0) wstat[warp][8 * n + 2 * c + j] = make_float2(m[n][j], sum);
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        float z = zs[n][y][j];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        float4 lo, hi;
        float* const a = &lo.x;
        float* const b = &hi.x;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float k = (t & 1) ? 0.0625f * up : up;
          a[t] = o[n][4 * y + t][j] * k * f + z;
          b[t] = o[n][4 * y + t][j + 2] * k * f + z;
        }
        float4* const to = reinterpret_cast<float4*>(to_rows + (8 * n + 2 * c + j) * D + 64 * y + 8 * g);
        to[0] = lo;
        to[1] = hi;
      }
    }
  __syncthreads();
  // ---- the CTA's rows: warps rw, rw + row_warps, ... hold the same rows of different positions
  const bool whole = passes == at.n;  // the item is all here: the result itself
  const int part = 2 * blockIdx.x + (at.pass == 0 ? 1 : 0);
  for (int k = threadIdx.x; k < r.p.row_warps * ROWS * (D / 4); k += kThreads) {
    const int rr = k / (D / 4), col = 4 * (k - rr * (D / 4)), w0 = rr / ROWS, wr = rr - w0 * ROWS;
    const int row = block_row + rr;
    if (row >= rows) break;
    float M = -INFINITY;
    for (int w = w0; w < kWarps; w += r.p.row_warps) M = fmaxf(M, wstat[w][wr].x);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    for (int w = w0; w < kWarps; w += r.p.row_warps) {
      const float2 st = wstat[w][wr];
      if (st.x == -INFINITY && st.y == 0.f) continue;
      const float e = exp2_fast(st.x - M);
      const float4 a = *reinterpret_cast<const float4*>(smem + (w * ROWS + wr) * D + col);
      L = fmaf(st.y, e, L);
      sum.x = fmaf(a.x, e, sum.x);
      sum.y = fmaf(a.y, e, sum.y);
      sum.z = fmaf(a.z, e, sum.z);
      sum.w = fmaf(a.w, e, sum.w);
    }
    if (whole) {
      const int token = s.q0 + row / group, head = h * group + row % group;
      const float inv = L == 0.f ? 0.f : 1.0f / L;
      const float y[4] = {sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv};
      store_f32<T, 4>(static_cast<T*>(r.a.out.ptr) + token * r.a.out.token_stride + head * r.a.out.head_stride + col, y);
    } else {
      const size_t to = (size_t)part * (r.p.row_warps * ROWS) + rr;
      *reinterpret_cast<float4*>(r.part + to * D + col) = sum;
      if (col == 0) r.stat[to] = make_float2(M, L);
    }
  }
  }
  now += passes;
  if (now >= last) return;
  __syncthreads();  // the ring is free again
  at.pass = 0;
  if (++at.unit == units) {
    at.unit = 0;
    do {
      ++at.i;
      at.n = passes_of(r, at.i);
    } while (at.n == 0);
  }
  }
}

// Joins the parts of one query row, CTA by CTA in ascending order within each of the thread groups and the
// groups in ascending order, so the result does not depend on timing.
template <typename T, int D>
__global__ void __launch_bounds__(D < 128 ? 128 : D) attn_join(const AttnRun r) {
  constexpr int LANES = D / 4, GROUPS = (D < 128 ? 128 : D) / LANES;
  __shared__ float4 sums[GROUPS][LANES];
  __shared__ float total_of[GROUPS];
  const int i = blockIdx.y, j = blockIdx.x / r.a.heads_q, head = blockIdx.x - j * r.a.heads_q;
  const Seq s = seq_of(r, i, false);
  const int group = r.a.heads_q / r.c.heads, h = head / group, units = r.c.heads * r.p.row_blocks;
  const int warp_lane = threadIdx.x & 31;
  const int per_block = r.p.row_warps * r.p.row_tiles * 8, row = j * group + (head - h * group);
  const int rb = row / per_block, rr = row - rb * per_block;
  // the item's passes [from, to) in the row of all, and the CTAs that have them
  long long before;
  const long long total = total_passes(r, warp_lane, i, &before) * units;
  const int n = passes_of(r, i);
  const long long from = before * units + (long long)(h * r.p.row_blocks + rb) * n, to = from + n;
  // Before any return: a launch that ends must not end before the one that it was set up beside.
  cudaGridDependencySynchronize();
  if (j >= min(s.nq, r.a.max_q)) return;
  const int of = sharers(r, total);
  int b0 = (int)(from * of / total);
  while (b0 > 0 && share_begin(total, b0, of) > from) --b0;
  while (share_begin(total, b0 + 1, of) <= from) ++b0;
  if (share_begin(total, b0 + 1, of) >= to) return;  // one CTA had it all and wrote the result
  int b1 = (int)((to - 1) * of / total);  // one past the last
  while (b1 > b0 && share_begin(total, b1, of) >= to) --b1;
  while (b1 < of && share_begin(total, b1, of) < to) ++b1;
  const int lane = threadIdx.x % LANES, part = threadIdx.x / LANES;
  // the first CTA has the item as its last one, all others as their first
  auto slot = [&](int b) { return ((size_t)2 * b + (b == b0 ? 1 : 0)) * per_block + rr; };
  float M = -INFINITY;
  for (int b = b0 + warp_lane; b < b1; b += 32) M = fmaxf(M, r.stat[slot(b)].x);
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f;
#pragma unroll 4
  for (int b = b0 + part; b < b1; b += GROUPS) {
    const float2 st = r.stat[slot(b)];
    const float e = st.x == -INFINITY && st.y == 0.f ? 0.f : exp2_fast(st.x - M);
    const float4 a = *reinterpret_cast<const float4*>(r.part + slot(b) * D + 4 * lane);
    L = fmaf(st.y, e, L);
    sum.x = fmaf(a.x, e, sum.x);
    sum.y = fmaf(a.y, e, sum.y);
    sum.z = fmaf(a.z, e, sum.z);
    sum.w = fmaf(a.w, e, sum.w);
  }
  sums[part][lane] = sum;
  if (lane == 0) total_of[part] = L;
  __syncthreads();
  if (part) return;
  for (int k = 1; k < GROUPS; ++k) {
    const float4 a = sums[k][lane];
    sum.x += a.x, sum.y += a.y, sum.z += a.z, sum.w += a.w;
    L += total_of[k];
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  const float y[4] = {sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv};
  store_f32<T, 4>(static_cast<T*>(r.a.out.ptr) + (s.q0 + j) * r.a.out.token_stride + head * r.a.out.head_stride + 4 * lane, y);
}

// Shared memory of a thread block: the rings and the queries' fragments, or the warps' results, after the last stage.
struct Shared {
  int q_offset, bytes;
};
constexpr Shared shared_of(int groups, int row_tiles, int terms, int row_warps) {
  const int dim = groups * 64, rings = kWarps / row_warps, stage = kStage * (dim + dim / 8);
  const int q_bytes = row_warps * row_tiles * 8 * (groups * terms * 128 + (groups + 1) * 4);
  const int out_bytes = kWarps * 8 * row_tiles * dim * 4, q_offset = rings * kStages * stage;
  return {q_offset, q_offset + q_bytes > out_bytes ? q_offset + q_bytes : out_bytes};
}

template <typename T, int NG, int NT>
cudaError_t run(const AttnRun& r, cudaStream_t st) {
  const auto kernel = attn_kernel<T, NG, NT>;
  // The limit belongs to the kernel, not to the call: always what its largest launch takes, so that a call of another
  // host thread never lowers it between this one's setting and launch.
  constexpr int terms = Held<T>::q, one = shared_of(NG, NT, terms, 1).bytes, two = shared_of(NG, NT, terms, 2).bytes,
                four = shared_of(NG, NT, terms, 4).bytes, most = one > two ? (one > four ? one : four) : two > four ? two : four;
  if (most > 32 * 1024) {  // with the static part, 48 KB need no leave
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  kernel<<<r.p.ctas, kThreads, r.p.smem, st>>>(r);
  return cudaGetLastError();
}

}  // namespace

AttnPlan plan_attn(const fmoe_kv_cache& c, const fmoe_attn_desc& a, int sms) {
  AttnPlan p;
  const long long rows = (long long)a.max_q * (a.heads_q / c.heads), tiles = (rows + 7) / 8;
  const int terms = terms_of(a.dtype), groups = c.dim / 64;
  // as few warps as can carry the rows, and then as few tiles a warp as that takes: what unpacking codes costs is
  // shared by more rows, and more warps have positions of their own. 12 requests of 5 queries, 4 heads a kv head of
  // 64, binary16: 40.5 us by three tiles of one warp, 47.2 by three warps; 16 heads a kv head of 256, 262144 positions:
  // 72.5 us by two tiles, 77.5 by two warps.
  const long long warps = (tiles + most_tiles(groups) - 1) / most_tiles(groups);
  p.row_tiles = (int)((tiles + warps - 1) / warps);
  p.row_warps = 1;
  while (p.row_warps < kWarps && p.row_warps < warps) p.row_warps *= 2;
  p.row_blocks = (int)((warps + p.row_warps - 1) / p.row_warps);
  const int at_once = resident(groups, p.row_tiles, terms);
  const int rings = kWarps / p.row_warps;
  const Shared shared = shared_of(groups, p.row_tiles, terms, p.row_warps);
  p.q_offset = shared.q_offset, p.smem = shared.bytes;
  const long long units = (long long)c.heads * p.row_blocks;
  const long long items = c.n_seqs * units, passes = std::max(1, (a.max_len + kStage - 1) / kStage);
  // Short sequences (kShort): a CTA takes one item, whatever its length, and nothing is left to join.
  // Else as many CTAs as are resident at once, or enough that every ring has a pass.
  p.by_item = passes <= kShort * rings;
  p.ctas = (int)(p.by_item ? items : std::min<long long>((items * passes + rings - 1) / rings, (long long)at_once * sms));
  p.ws_bytes = p.by_item ? 0 : (size_t)p.ctas * 2 * (p.row_warps * p.row_tiles * 8) * (c.dim * 4 + 8);
  return p;
}

cudaError_t launch_attn(const fmoe_kv_cache& c, const fmoe_attn_desc& a, const AttnPlan& p, void* ws, int* err,
                        cudaStream_t st, int* launches) {
  AttnRun r{c, a, p, static_cast<float*>(ws), nullptr, err};
  r.stat = reinterpret_cast<float2*>(r.part + (size_t)p.ctas * 2 * (p.row_warps * p.row_tiles * 8) * c.dim);
  return with_dtype(a.dtype, [&](auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    const int n = p.row_tiles;
    cudaError_t e = c.dim == 64    ? (n == 1   ? run<T, 1, 1>(r, st)
                                      : n == 2 ? run<T, 1, 2>(r, st)
                                      : n == 3 ? run<T, 1, 3>(r, st)
                                               : run<T, 1, 4>(r, st))
                    : c.dim == 128 ? (n == 1 ? run<T, 2, 1>(r, st) : n == 2 ? run<T, 2, 2>(r, st) : run<T, 2, 3>(r, st))
                                   : (n == 1 ? run<T, 4, 1>(r, st) : run<T, 4, 2>(r, st));
    if (e != cudaSuccess) return e;
    *launches = 1;
    if (!p.ws_bytes) return e;
    const dim3 grid(a.max_q * a.heads_q, c.n_seqs);
    const auto join = c.dim == 64 ? attn_join<T, 64> : c.dim == 128 ? attn_join<T, 128> : attn_join<T, 256>;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3(c.dim < 128 ? 128 : c.dim);
    config.stream = st;
    config.attrs = &early;
    config.numAttrs = 1;
    e = cudaLaunchKernelEx(&config, join, r);
    if (e == cudaSuccess) *launches = 2;
    return e;
  });
}

}  // namespace fmoe
