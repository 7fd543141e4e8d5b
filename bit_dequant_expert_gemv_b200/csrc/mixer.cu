// mixer.cu — the token mixers' part of the C ABI declared in include/fmoe.h: argument checks, scratch
// and launches (kernels in delta.cu, delta_chunk.cu, kv.cu, attn.cu).
#include "mixer.h"

#include <cmath>

#include "api.h"

using namespace fmoe;

namespace {

int element_bytes(int dtype) { return dtype == FMOE_F32 ? 4 : 2; }

int check_dtype(int dtype) {
  if (dtype != FMOE_F32 && dtype != FMOE_BF16 && dtype != FMOE_F16)
    return fail(FMOE_ERR_INVALID, "dtype %d is not FMOE_F32, FMOE_BF16 or FMOE_F16", dtype);
  return FMOE_OK;
}

int check_view(const char* name, const void* p, int64_t token_stride, int64_t head_stride, int dtype) {
  if (!p) return fail(FMOE_ERR_INVALID, "%s is NULL", name);
  if (token_stride < 0 || head_stride < 0) return fail(FMOE_ERR_INVALID, "%s has a negative stride", name);
  const int64_t per16 = 16 / element_bytes(dtype);
  if (!aligned16(p) || token_stride % per16 || head_stride % per16)
    return fail(FMOE_ERR_ALIGN, "%s and its strides must be multiples of 16 bytes", name);
  return FMOE_OK;
}

// Whether two of the rows [token][head] of `dim` elements share an element.
bool rows_overlap(int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride, int64_t head_stride) {
  if ((tokens > 1 && token_stride < dim) || (heads > 1 && head_stride < dim)) return true;
  if (tokens < 2 || heads < 2) return false;
  const __int128 ts = token_stride, hs = head_stride;
  if (ts >= (heads - 1) * hs + dim || hs >= (tokens - 1) * ts + dim) return false;  // one inside the other: the usual
  for (int64_t h = 1; h < heads; ++h) {  // strides that interleave: the tokens on either side of a head's offset
    const __int128 t = h * hs / ts, off = h * hs - t * ts;
    if ((t < tokens && off < dim) || (t + 1 < tokens && ts - off < dim)) return true;
  }
  return false;
}

int check_out(const char* name, const fmoe_out_view& v, int heads, int dim, int tokens, int dtype) {
  const int rc = check_view(name, v.ptr, v.token_stride, v.head_stride, dtype);
  if (rc) return rc;
  if (rows_overlap(tokens, heads, dim, v.token_stride, v.head_stride))
    return fail(FMOE_ERR_INVALID, "%s has overlapping rows", name);
  return FMOE_OK;
}

int check_delta(const fmoe_delta_desc* d, int n, int n_tokens) {
  if (!d) return fail(FMOE_ERR_INVALID, "descriptor is NULL");
  int rc = check_dtype(d->dtype);
  if (rc) return rc;
  if (d->heads_k < 1 || d->heads_v < 1 || d->heads_v % d->heads_k)
    return fail(FMOE_ERR_INVALID, "heads_v (%d) must be a positive multiple of heads_k (%d)", d->heads_v, d->heads_k);
  if ((d->dim_k != 64 && d->dim_k != 128) || (d->dim_v != 64 && d->dim_v != 128))
    return fail(FMOE_ERR_UNSUPPORTED, "dim_k (%d) and dim_v (%d) must be 64 or 128", d->dim_k, d->dim_v);
  if (d->heads_v > 65535) return fail(FMOE_ERR_UNSUPPORTED, "more than 65535 heads");
  if (n < 0 || n_tokens < 0) return fail(FMOE_ERR_INVALID, "negative count");
  if (n > (1 << 24)) return fail(FMOE_ERR_UNSUPPORTED, "more than %d sequences", 1 << 24);
  if ((long long)n * d->heads_v > 0x7fffffffll) return fail(FMOE_ERR_UNSUPPORTED, "more than 2^31 - 1 states in a call");
  if (d->n_slots < 0 || (!d->slots && d->n_slots < n))
    return fail(FMOE_ERR_INVALID, "%d state slots for %d sequences", d->n_slots, n);
  if (d->state_stride < (int64_t)d->heads_v * d->dim_k * d->dim_v || d->gate_stride < 0)
    return fail(FMOE_ERR_INVALID, "state_stride is smaller than a state, or gate_stride negative");
  if (!(d->eps >= 0.f)) return fail(FMOE_ERR_INVALID, "eps must be >= 0");
  if (n == 0 || n_tokens == 0) return FMOE_OK;
  if ((rc = check_view("q", d->q.ptr, d->q.token_stride, d->q.head_stride, d->dtype)) ||
      (rc = check_view("k", d->k.ptr, d->k.token_stride, d->k.head_stride, d->dtype)) ||
      (rc = check_view("v", d->v.ptr, d->v.token_stride, d->v.head_stride, d->dtype)) ||
      (rc = check_out("out", d->out, d->heads_v, d->dim_v, n_tokens, d->dtype)))
    return rc;
  if (!d->g || !d->beta || !d->state) return fail(FMOE_ERR_INVALID, "g, beta and state are required");
  if (!aligned16(d->state) || d->state_stride % 4)
    return fail(FMOE_ERR_ALIGN, "state and state_stride must be multiples of 16 bytes");
  return FMOE_OK;
}

int launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return cuda_fail(e, what);
  count_launch();
  return FMOE_OK;
}

int check_cache(const fmoe_kv_cache* c) {
  if (!c) return fail(FMOE_ERR_INVALID, "cache is NULL");
  if (c->dim != 64 && c->dim != 128 && c->dim != 256)
    return fail(FMOE_ERR_UNSUPPORTED, "dim (%d) must be 64, 128 or 256", c->dim);
  if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16)
    return fail(FMOE_ERR_UNSUPPORTED, "page_size (%d) must be a multiple of 16, at most 1024", c->page_size);
  if (c->heads < 1 || c->n_pages < 0 || c->n_seqs < 0 || c->max_pages < 0 || c->table_stride < 0)
    return fail(FMOE_ERR_INVALID, "cache has a negative count or stride, or no heads");
  if (c->heads > 65535) return fail(FMOE_ERR_UNSUPPORTED, "more than 65535 kv heads");
  if (c->n_pages > 0 && !c->pages) return fail(FMOE_ERR_INVALID, "pages is NULL");
  if (!aligned16(c->pages)) return fail(FMOE_ERR_ALIGN, "pages must be 16-byte aligned");
  if (c->n_seqs > 0 && c->max_pages > 0 && !c->page_table) return fail(FMOE_ERR_INVALID, "page_table is NULL");
  return FMOE_OK;
}

}  // namespace

extern "C" {

int fmoe_delta_step(const fmoe_delta_desc* d, int n, void* stream) {
  int rc = check_delta(d, n, n);
  if (rc || n == 0) return rc;
  DevState* dev;
  if ((rc = dev_state(&dev))) return rc;
  const DeltaRun r{*d, nullptr, nullptr, n, n, dev->err};
  return launched(launch_delta_recurrent(r, static_cast<cudaStream_t>(stream)), "delta step launch");
}

int fmoe_delta_chunk(const fmoe_delta_desc* d, const int32_t* cu_seqlens, int n, int n_tokens, int max_len,
                     const uint8_t* fresh, void* stream) {
  int rc = check_delta(d, n, n_tokens);
  if (rc) return rc;
  if (max_len < 0) return fail(FMOE_ERR_INVALID, "max_len is negative");
  if (n == 0 || n_tokens == 0) return FMOE_OK;
  if (!cu_seqlens) return fail(FMOE_ERR_INVALID, "cu_seqlens is NULL");
  DevState* dev;
  if ((rc = dev_state(&dev))) return rc;
  const DeltaRun r{*d, cu_seqlens, fresh, n, n_tokens, dev->err};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // A chunk costs as much however few of its 64 tokens there are. Recurrent and chunked form in us, 32 heads of
  // 128 x 128: sequences of 8 tokens 9.6 and 15.0 (one), 27 and 30 (8 of them), 191 and 225 (64); of 16 tokens
  // 16.4 and 15.7, 50 and 29, 352 and 226; of 64 tokens 57 and 16, 190 and 33, 1322 and 230.
  const bool chunked = d->dtype != FMOE_F32 && max_len >= 16;
  return launched(chunked ? launch_delta_chunk(r, st) : launch_delta_recurrent(r, st), "delta chunk launch");
}

size_t fmoe_kv_block_bytes(int page_size, int dim) {
  if (page_size < 16 || page_size > 1024 || page_size % 16 || (dim != 64 && dim != 128 && dim != 256)) return 0;
  return (size_t)page_size * (size_t)(dim + dim / 8);
}

int fmoe_kv_append(const fmoe_kv_cache* cache, const fmoe_kv_tokens* t, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (!t) return fail(FMOE_ERR_INVALID, "tokens is NULL");
  if ((rc = check_dtype(t->dtype))) return rc;
  if ((long long)t->n_tokens * (t->heads_q + 2ll * cache->heads) > (1ll << 33))
    return fail(FMOE_ERR_UNSUPPORTED, "more than 2^33 rows");
  if (t->n_tokens < 0 || t->heads_q < 0 || t->n_freq < 0 || t->n_freq > cache->dim / 2)
    return fail(FMOE_ERR_INVALID, "negative count, or n_freq (%d) above dim / 2", t->n_freq);
  if (t->n_tokens == 0) return FMOE_OK;
  if ((rc = check_view("k", t->k.ptr, t->k.token_stride, t->k.head_stride, t->dtype)) ||
      (rc = check_view("v", t->v.ptr, t->v.token_stride, t->v.head_stride, t->dtype)))
    return rc;
  if (t->heads_q > 0 &&
      ((rc = check_view("q", t->q.ptr, t->q.token_stride, t->q.head_stride, t->dtype)) ||
       (rc = check_out("q_out", t->q_out, t->heads_q, cache->dim, t->n_tokens, t->dtype))))
    return rc;
  if (!t->positions || (t->n_freq > 0 && !t->inv_freq))
    return fail(FMOE_ERR_INVALID, "positions and inv_freq are required");
  if (t->heads_q > 0 && t->q_out.ptr == t->q.ptr &&
      (t->q_out.token_stride != t->q.token_stride || t->q_out.head_stride != t->q.head_stride))
    return fail(FMOE_ERR_INVALID, "q_out is q but has other strides");
  DevState* dev;
  if ((rc = dev_state(&dev))) return rc;
  return launched(launch_kv_append(*cache, *t, dev->sms, dev->err, static_cast<cudaStream_t>(stream)), "append launch");
}

int fmoe_kv_read(const fmoe_kv_cache* cache, const int32_t* positions, const int32_t* seq, int n_tokens, int dtype,
                 fmoe_out_view k_out, fmoe_out_view v_out, void* stream) {
  int rc = check_cache(cache);
  if (rc || (rc = check_dtype(dtype))) return rc;
  if (n_tokens < 0) return fail(FMOE_ERR_INVALID, "negative count");
  if (n_tokens * 2ll * cache->heads > (1ll << 33)) return fail(FMOE_ERR_UNSUPPORTED, "more than 2^33 rows");
  if (n_tokens == 0) return FMOE_OK;
  if ((rc = check_out("k_out", k_out, cache->heads, cache->dim, n_tokens, dtype)) ||
      (rc = check_out("v_out", v_out, cache->heads, cache->dim, n_tokens, dtype)))
    return rc;
  if (!positions) return fail(FMOE_ERR_INVALID, "positions is NULL");
  DevState* dev;
  if ((rc = dev_state(&dev))) return rc;
  return launched(launch_kv_read(*cache, positions, seq, n_tokens, dtype, k_out, v_out, dev->err,
                                 static_cast<cudaStream_t>(stream)),
                  "read launch");
}

int fmoe_attn_q4(const fmoe_kv_cache* cache, const fmoe_attn_desc* a, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (!a) return fail(FMOE_ERR_INVALID, "descriptor is NULL");
  if ((rc = check_dtype(a->dtype))) return rc;
  if (a->heads_q < 1 || a->heads_q % cache->heads)
    return fail(FMOE_ERR_INVALID, "heads_q (%d) must be a positive multiple of the cache's heads (%d)", a->heads_q,
                cache->heads);
  if (a->n_tokens < 0 || a->max_q < 0 || a->max_len < 0) return fail(FMOE_ERR_INVALID, "negative count");
  if (!std::isfinite(a->scale)) return fail(FMOE_ERR_INVALID, "scale is not finite");
  if (!a->cu_q && a->n_tokens != cache->n_seqs)
    return fail(FMOE_ERR_INVALID, "%d queries for %d sequences without cu_q", a->n_tokens, cache->n_seqs);
  if (a->n_tokens == 0 || cache->n_seqs == 0) return FMOE_OK;
  if (a->max_q == 0) return fail(FMOE_ERR_INVALID, "max_q is 0 with %d queries", a->n_tokens);
  if ((rc = check_view("q", a->q.ptr, a->q.token_stride, a->q.head_stride, a->dtype)) ||
      (rc = check_out("out", a->out, a->heads_q, cache->dim, a->n_tokens, a->dtype)))
    return rc;
  if (!a->lens) return fail(FMOE_ERR_INVALID, "lens is NULL");
  if (cache->n_seqs > 65535) return fail(FMOE_ERR_UNSUPPORTED, "more than 65535 sequences");
  if ((long long)a->max_q * a->heads_q > (1 << 30) || a->max_len > (1 << 30))
    return fail(FMOE_ERR_UNSUPPORTED, "max_q * heads_q or max_len above 2^30");
  DevState* dev;
  if ((rc = dev_state(&dev))) return rc;
  const AttnPlan p = plan_attn(*cache, *a, dev->sms);
  if ((long long)cache->heads * p.row_blocks > 65535 || (long long)cache->n_seqs * cache->heads * p.row_blocks > (1 << 30))
    return fail(FMOE_ERR_UNSUPPORTED, "too many query rows of a sequence (max_q %d)", a->max_q);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  if (p.ws_bytes) {
    const cudaError_t e = cudaMallocFromPoolAsync(&ws, p.ws_bytes, dev->pool, st);
    if (e != cudaSuccess) return fail(FMOE_ERR_NOMEM, "scratch allocation: %s", cudaGetErrorString(e));
  }
  int launches = 0;
  const cudaError_t e = launch_attn(*cache, *a, p, ws, dev->err, st, &launches);
  for (int i = 0; i < launches; ++i) count_launch();
  const cudaError_t e2 = ws ? cudaFreeAsync(ws, st) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  if (e2 != cudaSuccess) return cuda_fail(e2, "scratch free");
  return FMOE_OK;
}

}  // extern "C"
