// C entry points over uncompressed keys and values: tpla_kv_append,
// tpla_kv_decode, tpla_kv_prefill (argument checks, workspaces, launches).
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "internal.h"
#include "tpla.h"

namespace tpla {
namespace {

constexpr int64_t kMaxBatch = 1 << 20;
constexpr int kMaxHeads = 4096;
constexpr int64_t kMaxPagesRow = 1 << 24;
constexpr int64_t kMaxRows = 1 << 30;  // tokens of a request, rows of a packed tensor

bool is16(int dtype) { return dtype == TPLA_BF16 || dtype == TPLA_F16; }

bool empty(const tpla_tensor* t) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] == 0) return true;
  return false;
}

// Rows on 16-byte boundaries, every dimension of more than one entry with a
// stride of its own (a broadcast dimension has no tensor map, and rows that
// are written must not lie over one another).
bool rows16(const tpla_tensor* t) {
  if (empty(t)) return true;
  const int64_t esz = is16(t->dtype) ? 2 : 4;
  if (!aligned16(t->data)) return false;
  for (int i = 0; i + 1 < t->ndim; ++i) {
    if (t->shape[i] > 1 && (t->stride[i] * esz % 16 || t->stride[i] == 0)) return false;
  }
  return true;
}

// Largest stride in bytes that a tensor map takes is below 2^40.
bool map_strides(const tpla_tensor* t) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->stride[i] >= (1LL << 38)) return false;
  return true;
}

// The caches of an append or an attention call and the page table that maps
// requests to them (B requests).
int check_caches(const tpla_tensor* k, const tpla_tensor* v, const tpla_tensor* page_table,
                 int64_t B, int64_t* cap_rows) {
  if (!k || !is16(k->dtype) || !check_tensor(k, k->dtype, 4) || !rows16(k))
    return TPLA_ERR_INVALID_ARG;
  if (v) {
    if (v->dtype != k->dtype || !check_tensor(v, k->dtype, 4) || !rows16(v))
      return TPLA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
      if (v->shape[i] != k->shape[i]) return TPLA_ERR_INVALID_ARG;
  }
  if (page_table) {
    if (!check_tensor(page_table, TPLA_I32, 2) || page_table->shape[0] != B)
      return TPLA_ERR_INVALID_ARG;
    if (k->shape[1] != kBlock) return TPLA_ERR_UNSUPPORTED;  // 64-token pages only
    if (page_table->shape[1] < 1 && B > 0) return TPLA_ERR_INVALID_ARG;
    if (page_table->shape[1] > kMaxPagesRow) return TPLA_ERR_UNSUPPORTED;
    *cap_rows = page_table->shape[1] * kBlock;
  } else {
    if (k->shape[0] != B) return TPLA_ERR_INVALID_ARG;
    *cap_rows = k->shape[1];
  }
  if (k->shape[0] >= (1LL << 31) - 1 || k->shape[2] > kMaxHeads || *cap_rows > kMaxRows)
    return TPLA_ERR_UNSUPPORTED;
  return TPLA_OK;
}

int build_append(const tpla_tensor* k, const tpla_tensor* v, const tpla_tensor* positions,
                 const tpla_tensor* requests, const tpla_tensor* pt, const tpla_tensor* kc,
                 const tpla_tensor* vc, const tpla_tensor* cs, int rope_offset, int interleaved,
                 const tpla_tensor* q, const tpla_tensor* qo, int q_rope_offset,
                 KvAppendProblem* p) {
  memset(p, 0, sizeof(*p));
  if (!k || !kc || !is16(kc->dtype)) return TPLA_ERR_INVALID_ARG;
  if (k->dtype != TPLA_F32 && k->dtype != kc->dtype) return TPLA_ERR_INVALID_ARG;
  if (!check_tensor(k, k->dtype, 3) || !rows16(k)) return TPLA_ERR_INVALID_ARG;
  const int64_t T = k->shape[0], Hkv = k->shape[1], Dk = k->shape[2];
  if (!check_tensor(positions, TPLA_I32, 1) || positions->shape[0] != T)
    return TPLA_ERR_INVALID_ARG;
  if (requests && (!check_tensor(requests, TPLA_I32, 1) || requests->shape[0] != T))
    return TPLA_ERR_INVALID_ARG;
  if (T > 0 && (positions->stride[0] != 1 || (requests && requests->stride[0] != 1)) && T > 1)
    return TPLA_ERR_INVALID_ARG;
  // without `requests` token t belongs to request t; with it the number of
  // requests is the page table's (or the contiguous cache's)
  const int64_t B = requests ? (pt ? pt->shape[0] : kc->shape[0]) : T;
  if ((v == nullptr) != (vc == nullptr)) return TPLA_ERR_INVALID_ARG;
  int64_t cap = 0;
  int rc = check_caches(kc, vc, pt, B, &cap);
  if (rc != TPLA_OK) return rc;
  if (kc->shape[2] != Hkv || kc->shape[3] != Dk || Dk < 8 || Dk % 8) return TPLA_ERR_INVALID_ARG;
  if (v) {
    if (v->dtype != k->dtype || !check_tensor(v, k->dtype, 3) || !rows16(v) ||
        v->shape[0] != T || v->shape[1] != Hkv || v->shape[2] != vc->shape[3] ||
        v->shape[2] < 8 || v->shape[2] % 8)
      return TPLA_ERR_INVALID_ARG;
  }
  int64_t rot = 0;
  if (cs) {
    if (!check_tensor(cs, TPLA_F32, 2) || !rows16(cs)) return TPLA_ERR_INVALID_ARG;
    rot = cs->shape[1];
    if (rot < 16 || rot % 16 || !(interleaved == 0 || interleaved == 1))
      return TPLA_ERR_INVALID_ARG;
    if (rope_offset < 0 || rope_offset % 8 || rope_offset + rot > Dk) return TPLA_ERR_INVALID_ARG;
  }
  if (q) {
    if (!cs || !qo || qo->dtype != kc->dtype) return TPLA_ERR_INVALID_ARG;
    if (q->dtype != TPLA_F32 && q->dtype != kc->dtype) return TPLA_ERR_INVALID_ARG;
    if (!check_tensor(q, q->dtype, 3) || !check_tensor(qo, qo->dtype, 3) || !rows16(q) ||
        !rows16(qo) || q->shape[0] != T)
      return TPLA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
      if (q->shape[i] != qo->shape[i]) return TPLA_ERR_INVALID_ARG;
    if (q->shape[2] % 8 || q_rope_offset < 0 || q_rope_offset % 8 ||
        q_rope_offset + rot > q->shape[2])
      return TPLA_ERR_INVALID_ARG;
    // in place only where every row is its own destination
    if (q->data == qo->data && T > 0 &&
        (q->dtype != qo->dtype || (T > 1 && q->stride[0] != qo->stride[0]) ||
         (q->shape[1] > 1 && q->stride[1] != qo->stride[1])))
      return TPLA_ERR_INVALID_ARG;
  } else if (qo) {
    return TPLA_ERR_INVALID_ARG;
  }
  if (T > kMaxRows || B > kMaxBatch || Hkv > kMaxHeads || (q && q->shape[1] > kMaxHeads) ||
      Dk > 4096 || (v && v->shape[2] > 4096) || (q && q->shape[2] > 4096))
    return TPLA_ERR_UNSUPPORTED;
  p->k = k->data;
  p->k_st = k->stride[0];
  p->k_sh = k->stride[1];
  p->kv_f32 = k->dtype == TPLA_F32;
  p->k_cache = kc->data;
  p->kc_s0 = kc->stride[0];
  p->kc_s1 = kc->stride[1];
  p->kc_s2 = kc->stride[2];
  p->rot = (int)rot;
  p->interleaved = interleaved;
  auto pieces = [&](int64_t width, bool rotated) {
    if (!rotated) return (int)(width / 8);
    return (int)((width - rot) / 8 + (interleaved ? rot / 8 : rot / 16));
  };
  p->k_off = rope_offset;
  p->k_pieces = pieces(Dk, cs != nullptr);
  if (v) {
    p->v = v->data;
    p->v_st = v->stride[0];
    p->v_sh = v->stride[1];
    p->v_cache = vc->data;
    p->vc_s0 = vc->stride[0];
    p->vc_s1 = vc->stride[1];
    p->vc_s2 = vc->stride[2];
    p->v_pieces = pieces(v->shape[2], false);
  }
  if (q) {
    p->q = q->data;
    p->q_st = q->stride[0];
    p->q_sh = q->stride[1];
    p->q_f32 = q->dtype == TPLA_F32;
    p->q_out = qo->data;
    p->qo_st = qo->stride[0];
    p->qo_sh = qo->stride[1];
    p->q_off = q_rope_offset;
    p->q_pieces = pieces(q->shape[2], true);
    p->Hq = (int)q->shape[1];
  }
  p->num_blocks = kc->shape[0];
  p->cap_rows = cap;
  p->positions = reinterpret_cast<const int*>(positions->data);
  p->requests = requests ? reinterpret_cast<const int*>(requests->data) : nullptr;
  p->page_table = pt ? reinterpret_cast<const int*>(pt->data) : nullptr;
  p->pt_sb = pt ? pt->stride[0] : 0;
  p->B = (int)B;
  p->cos_sin = cs ? reinterpret_cast<const float*>(cs->data) : nullptr;
  p->cs_s = cs ? cs->stride[0] : 0;
  p->table_rows = cs ? cs->shape[0] : 0;
  p->T = (int)T;
  p->Hkv = (int)Hkv;
  p->f16 = kc->dtype == TPLA_F16;
  return TPLA_OK;
}

// out and lse of an attention call with `rows` query rows of Hq heads.
int check_results(const tpla_tensor* out, const tpla_tensor* lse, int dtype, int64_t rows,
                  int64_t Hq, int64_t Dv) {
  if (!out || (out->dtype != TPLA_F32 && out->dtype != dtype)) return TPLA_ERR_INVALID_ARG;
  if (!check_tensor(out, out->dtype, 3) || !rows16(out) || out->shape[0] != rows ||
      out->shape[1] != Hq || out->shape[2] != Dv)
    return TPLA_ERR_INVALID_ARG;
  if (lse && (!check_tensor(lse, TPLA_F32, 3) || lse->shape[0] != rows || lse->shape[1] != Hq ||
              lse->shape[2] != 1 || (rows > 1 && lse->stride[0] == 0) ||
              (Hq > 1 && lse->stride[1] == 0)))
    return TPLA_ERR_INVALID_ARG;
  return TPLA_OK;
}

// The kernels work in log2 units: scale log2(e) has to be an f32 too.
bool check_scale(float scale) { return isfinite((float)(scale * 1.4426950408889634)); }

// Queries [rows, Hq, Dk] against Hkv heads of Dk and Dv columns.
int check_heads(const tpla_tensor* q, int dtype, int64_t Hkv, int64_t Dk, int64_t Dv) {
  if (!q || q->dtype != dtype || !check_tensor(q, dtype, 3) || !rows16(q) || q->shape[2] != Dk)
    return TPLA_ERR_INVALID_ARG;
  if (Hkv < 1 || q->shape[1] < 1 || q->shape[1] % Hkv) return TPLA_ERR_INVALID_ARG;
  if (q->shape[1] > kMaxHeads || !kv_head_dims_supported((int)Dk, (int)Dv))
    return TPLA_ERR_UNSUPPORTED;
  return TPLA_OK;
}

void fill_cache_source(const tpla_tensor* k, const tpla_tensor* v, const tpla_tensor* pt,
                       const tpla_tensor* seq, int64_t cap, KvSource* s) {
  s->k = k->data;
  s->v = v->data;
  s->k_s0 = k->stride[0];
  s->k_s1 = k->stride[1];
  s->k_s2 = k->stride[2];
  s->v_s0 = v->stride[0];
  s->v_s1 = v->stride[1];
  s->v_s2 = v->stride[2];
  s->num_blocks = k->shape[0];
  s->cap_rows = cap;
  s->seq_lens = reinterpret_cast<const int*>(seq->data);
  s->page_table = pt ? reinterpret_cast<const int*>(pt->data) : nullptr;
  s->pt_sb = pt ? pt->stride[0] : 0;
  s->Hkv = (int)k->shape[2];
  s->Dk = (int)k->shape[3];
  s->Dv = (int)v->shape[3];
  s->f16 = k->dtype == TPLA_F16;
}

int build_decode(const tpla_tensor* q, const tpla_tensor* k, const tpla_tensor* v,
                 const tpla_tensor* seq, const tpla_tensor* pt, float scale,
                 const tpla_tensor* out, const tpla_tensor* lse, KvDecodeProblem* p) {
  memset(p, 0, sizeof(*p));
  if (!q || !k || !v || !check_scale(scale)) return TPLA_ERR_INVALID_ARG;
  const int64_t B = q->ndim == 3 ? q->shape[0] : -1;
  if (B > kMaxBatch) return TPLA_ERR_UNSUPPORTED;
  int64_t cap = 0;
  int rc = check_caches(k, v, pt, B, &cap);
  if (rc != TPLA_OK) return rc;
  if (!map_strides(k) || !map_strides(v)) return TPLA_ERR_UNSUPPORTED;
  rc = check_heads(q, k->dtype, k->shape[2], k->shape[3], v->shape[3]);
  if (rc != TPLA_OK) return rc;
  if (!check_tensor(seq, TPLA_I32, 1) || seq->shape[0] != B || (B > 1 && seq->stride[0] != 1))
    return TPLA_ERR_INVALID_ARG;
  rc = check_results(out, lse, k->dtype, B, q->shape[1], v->shape[3]);
  if (rc != TPLA_OK) return rc;
  if (B * q->shape[1] > (1LL << 30)) return TPLA_ERR_UNSUPPORTED;
  fill_cache_source(k, v, pt, seq, cap, &p->kv);
  p->q = q->data;
  p->q_sb = q->stride[0];
  p->q_sh = q->stride[1];
  p->B = (int)B;
  p->Hq = (int)q->shape[1];
  p->scale = scale;
  p->out = out->data;
  p->out_dtype = out->dtype;
  p->o_sb = out->stride[0];
  p->o_sh = out->stride[1];
  p->lse = lse ? reinterpret_cast<float*>(lse->data) : nullptr;
  p->l_sb = lse ? lse->stride[0] : 0;
  p->l_sh = lse ? lse->stride[1] : 0;
  return TPLA_OK;
}

int build_kv_prefill(const tpla_tensor* q, const tpla_tensor* k, const tpla_tensor* v,
                     const tpla_tensor* cu_q, const tpla_tensor* cu_k, const tpla_tensor* seq,
                     const tpla_tensor* pt, int causal, float scale, const tpla_tensor* out,
                     const tpla_tensor* lse, KvPrefillProblem* p) {
  memset(p, 0, sizeof(*p));
  if (!q || !k || !v || !check_scale(scale) || !(causal == 0 || causal == 1))
    return TPLA_ERR_INVALID_ARG;
  if (!check_tensor(cu_q, TPLA_I32, 1) || cu_q->shape[0] < 1 ||
      (cu_q->shape[0] > 1 && cu_q->stride[0] != 1))
    return TPLA_ERR_INVALID_ARG;
  const int64_t B = cu_q->shape[0] - 1;
  if (B > kMaxBatch) return TPLA_ERR_UNSUPPORTED;
  int rc;
  if (pt) {
    int64_t cap = 0;
    rc = check_caches(k, v, pt, B, &cap);
    if (rc != TPLA_OK) return rc;
    if (cu_k || !check_tensor(seq, TPLA_I32, 1) || seq->shape[0] != B ||
        (B > 1 && seq->stride[0] != 1))
      return TPLA_ERR_INVALID_ARG;
    fill_cache_source(k, v, pt, seq, cap, &p->kv);
  } else {
    if (seq || !is16(k->dtype) || v->dtype != k->dtype || !check_tensor(k, k->dtype, 3) ||
        !check_tensor(v, k->dtype, 3) || !rows16(k) || !rows16(v) ||
        k->shape[0] != v->shape[0] || k->shape[1] != v->shape[1])
      return TPLA_ERR_INVALID_ARG;
    if (cu_k && (!check_tensor(cu_k, TPLA_I32, 1) || cu_k->shape[0] != B + 1 ||
                 (B > 0 && cu_k->stride[0] != 1)))
      return TPLA_ERR_INVALID_ARG;
    if (k->shape[0] > kMaxRows || k->shape[1] > kMaxHeads) return TPLA_ERR_UNSUPPORTED;
    KvSource& s = p->kv;
    s.k = k->data;
    s.v = v->data;
    s.k_s1 = k->stride[0];
    s.k_s2 = k->stride[1];
    s.v_s1 = v->stride[0];
    s.v_s2 = v->stride[1];
    s.num_blocks = 1;
    s.cap_rows = k->shape[0];
    s.Hkv = (int)k->shape[1];
    s.Dk = (int)k->shape[2];
    s.Dv = (int)v->shape[2];
    s.f16 = k->dtype == TPLA_F16;
    p->cu_k = reinterpret_cast<const int*>(cu_k ? cu_k->data : cu_q->data);
  }
  if (!map_strides(k) || !map_strides(v) || !map_strides(q)) return TPLA_ERR_UNSUPPORTED;
  rc = check_heads(q, k->dtype, p->kv.Hkv, p->kv.Dk, p->kv.Dv);
  if (rc != TPLA_OK) return rc;
  rc = check_results(out, lse, k->dtype, q->shape[0], q->shape[1], p->kv.Dv);
  if (rc != TPLA_OK) return rc;
  if (q->shape[0] > kMaxRows || q->shape[0] * q->shape[1] > (1LL << 40)) return TPLA_ERR_UNSUPPORTED;
  p->q = q->data;
  p->q_st = q->stride[0];
  p->q_sh = q->stride[1];
  p->cu_q = reinterpret_cast<const int*>(cu_q->data);
  p->B = (int)B;
  p->T = (int)q->shape[0];
  p->Hq = (int)q->shape[1];
  p->causal = causal;
  p->scale = scale;
  p->out = out->data;
  p->out_dtype = out->dtype;
  p->o_st = out->stride[0];
  p->o_sh = out->stride[1];
  p->lse = lse ? reinterpret_cast<float*>(lse->data) : nullptr;
  p->l_st = lse ? lse->stride[0] : 0;
  p->l_sh = lse ? lse->stride[1] : 0;
  return TPLA_OK;
}

// Runs `launch(workspace)` with the caller's workspace or, where that is
// NULL, one of the stream-ordered allocator.
template <typename F>
int with_workspace(void* ws, size_t have, size_t need, cudaStream_t s, F launch) {
  if (ws && (have < need || !aligned16(ws))) return TPLA_ERR_WORKSPACE;
  bool owned = false;
  if (!ws && need > 0) {
    cudaError_t e = cudaMallocAsync(&ws, need, s);
    if (e != cudaSuccess) return cuda_fail(e);
    owned = true;
  }
  cudaError_t e = launch(ws);
  int rc = e == cudaSuccess ? TPLA_OK : cuda_fail(e);
  if (owned) {
    e = cudaFreeAsync(ws, s);
    if (rc == TPLA_OK && e != cudaSuccess) rc = cuda_fail(e);
  }
  return rc;
}

}  // namespace

int sm_count(int device) {
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
      sms < 1) {
    cudaGetLastError();
    sms = 148;  // no device: the workspace sizes of a B200
  }
  return sms;
}

}  // namespace tpla

using namespace tpla;

extern "C" {

int tpla_kv_append(const tpla_tensor* k_new, const tpla_tensor* v_new,
                   const tpla_tensor* positions, const tpla_tensor* requests,
                   const tpla_tensor* page_table, tpla_tensor* k_cache, tpla_tensor* v_cache,
                   const tpla_tensor* cos_sin, int rope_offset, int interleaved,
                   const tpla_tensor* q, tpla_tensor* q_out, int q_rope_offset,
                   tpla_stream_t stream) {
  KvAppendProblem p;
  int rc = build_append(k_new, v_new, positions, requests, page_table, k_cache, v_cache, cos_sin,
                        rope_offset, interleaved, q, q_out, q_rope_offset, &p);
  if (rc != TPLA_OK) return rc;
  cudaError_t e = launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? TPLA_OK : cuda_fail(e);
}

int tpla_kv_decode_workspace_size(const tpla_tensor* q, const tpla_tensor* k_cache,
                                  const tpla_tensor* v_cache, const tpla_tensor* page_table,
                                  size_t* bytes) {
  if (!bytes || !q || !k_cache || !v_cache) return TPLA_ERR_INVALID_ARG;
  const int64_t B = q->ndim == 3 ? q->shape[0] : -1;
  if (B > kMaxBatch) return TPLA_ERR_UNSUPPORTED;
  int64_t cap = 0;
  int rc = check_caches(k_cache, v_cache, page_table, B, &cap);
  if (rc != TPLA_OK) return rc;
  rc = check_heads(q, k_cache->dtype, k_cache->shape[2], k_cache->shape[3], v_cache->shape[3]);
  if (rc != TPLA_OK) return rc;
  KvDecodeProblem p;
  memset(&p, 0, sizeof(p));
  p.kv.cap_rows = cap;
  p.kv.Hkv = (int)k_cache->shape[2];
  p.kv.Dv = (int)v_cache->shape[3];
  p.B = (int)B;
  p.Hq = (int)q->shape[1];
  *bytes = B > 0 ? kv_decode_workspace_bytes(p, current_device()) : 0;
  return TPLA_OK;
}

int tpla_kv_decode(const tpla_tensor* q, const tpla_tensor* k_cache, const tpla_tensor* v_cache,
                   const tpla_tensor* seq_lens, const tpla_tensor* page_table, float scale,
                   tpla_tensor* out, tpla_tensor* lse, void* workspace, size_t workspace_bytes,
                   tpla_stream_t stream) {
  KvDecodeProblem p;
  int rc = build_decode(q, k_cache, v_cache, seq_lens, page_table, scale, out, lse, &p);
  if (rc != TPLA_OK) return rc;
  if (p.B == 0) return TPLA_OK;
  if (!sm100_device(current_device())) return TPLA_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return with_workspace(workspace, workspace_bytes, kv_decode_workspace_bytes(p, current_device()),
                        s, [&](void* ws) { return launch_kv_decode(p, ws, s); });
}

int tpla_kv_prefill_workspace_size(const tpla_tensor* q, const tpla_tensor* k,
                                   const tpla_tensor* v, const tpla_tensor* cu_q,
                                   const tpla_tensor* page_table, size_t* bytes) {
  if (!bytes || !q || !k || !v || !cu_q || q->ndim != 3 || cu_q->ndim != 1 ||
      cu_q->shape[0] < 1 || k->ndim != (page_table ? 4 : 3) || v->ndim != k->ndim ||
      (page_table && page_table->ndim != 2))
    return TPLA_ERR_INVALID_ARG;
  const int64_t Hkv = k->shape[k->ndim - 2], Dv = v->shape[v->ndim - 1];
  const int64_t cap = page_table ? page_table->shape[1] * kBlock : k->shape[0];
  if (q->shape[0] < 0 || Hkv < 1 || q->shape[1] < 1 || q->shape[1] % Hkv || Dv < 1 || cap < 0)
    return TPLA_ERR_INVALID_ARG;
  if (q->shape[0] > kMaxRows || q->shape[1] > kMaxHeads || cu_q->shape[0] - 1 > kMaxBatch ||
      cap > kMaxRows || Dv > 4096)
    return TPLA_ERR_UNSUPPORTED;
  KvPrefillProblem p;
  memset(&p, 0, sizeof(p));
  p.kv.Hkv = (int)Hkv;
  p.kv.Dv = (int)Dv;
  p.kv.cap_rows = cap;
  p.T = (int)q->shape[0];
  p.Hq = (int)q->shape[1];
  p.B = (int)cu_q->shape[0] - 1;
  *bytes = p.T > 0 && p.B > 0 ? kv_prefill_workspace_bytes(p) : 0;
  return TPLA_OK;
}

int tpla_kv_prefill(const tpla_tensor* q, const tpla_tensor* k, const tpla_tensor* v,
                    const tpla_tensor* cu_q, const tpla_tensor* cu_k, const tpla_tensor* seq_lens,
                    const tpla_tensor* page_table, int causal, float scale, tpla_tensor* out,
                    tpla_tensor* lse, void* workspace, size_t workspace_bytes,
                    tpla_stream_t stream) {
  KvPrefillProblem p;
  int rc = build_kv_prefill(q, k, v, cu_q, cu_k, seq_lens, page_table, causal, scale, out, lse, &p);
  if (rc != TPLA_OK) return rc;
  if (p.B == 0 || p.T == 0) return TPLA_OK;
  if (!sm100_device(current_device())) return TPLA_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return with_workspace(workspace, workspace_bytes, kv_prefill_workspace_bytes(p), s,
                        [&](void* ws) { return launch_kv_prefill(p, ws, s); });
}

}  // extern "C"
