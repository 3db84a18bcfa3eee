// Append of uncompressed keys and values to a paged (or contiguous) cache,
// with the rotary position embedding on the way, and of the same rotation on
// the queries of the same tokens.
//
// A token at position p turns the pairs (a_j, b_j), j < n, of the rotated
// columns by the table's angles:
//   a' = a cos[p][j] - b sin[p][j],   b' = b cos[p][j] + a sin[p][j]
// The pairs are columns (off + j, off + n + j) (halves) or (off + 2j,
// off + 2j + 1) (interleaved); the other columns pass through.  Arithmetic is
// f32, with one rounding to the cache's 16-bit type.
//
// Nothing is reused but the table row, so the bytes bound it: every value is
// read once and written once in 16-byte pieces (8 values).  A thread owns
// both halves of its pairs, so queries may be rotated in place.
#include <stdint.h>

#include "internal.h"
#include "kv_ptx.cuh"

namespace tpla {
namespace {

using namespace kvx;

__device__ int g_kv_append_status;

constexpr int kThreads = 256;

// 8 consecutive values as f32
template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t off, bool f32, float (&x)[8]) {
  if (f32) {
    const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + off);
    const float4 a = s[0], b = s[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + off);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = T::unpack(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(uint16_t* dst, const float (&x)[8]) {
  uint4 v;
  v.x = T::pack(x[0], x[1]);
  v.y = T::pack(x[2], x[3]);
  v.z = T::pack(x[4], x[5]);
  v.w = T::pack(x[6], x[7]);
  *reinterpret_cast<uint4*>(dst) = v;
}

// Piece i of a row of `width` columns: the pieces of rotated pairs first
// (two halves of 8 columns, or 8 interleaved columns), then plain copies.
template <typename T>
__device__ __forceinline__ void row_piece(const void* src, int64_t s_off, bool f32, uint16_t* dst,
                                          int i, int rot, int off, bool inter, const float* cs) {
  float x[8];
  const int n = rot >> 1;
  const int pieces = inter ? rot >> 3 : rot >> 4;
  if (i >= pieces) {  // a plain copy
    int c = (i - pieces) << 3;
    if (c >= off) c += rot;
    load8<T>(src, s_off + c, f32, x);
    store8<T>(dst + c, x);
    return;
  }
  if (inter) {
    const int c = off + (i << 3);
    load8<T>(src, s_off + c, f32, x);
    const float4 co = *reinterpret_cast<const float4*>(cs + 4 * i);
    const float4 si = *reinterpret_cast<const float4*>(cs + n + 4 * i);
    const float cv[4] = {co.x, co.y, co.z, co.w}, sv[4] = {si.x, si.y, si.z, si.w};
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[2 * j] = x[2 * j] * cv[j] - x[2 * j + 1] * sv[j];
      y[2 * j + 1] = x[2 * j + 1] * cv[j] + x[2 * j] * sv[j];
    }
    store8<T>(dst + c, y);
    return;
  }
  const int c = off + (i << 3);
  float z[8];
  load8<T>(src, s_off + c, f32, x);
  load8<T>(src, s_off + c + n, f32, z);
  float cv[8], sv[8];
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    *reinterpret_cast<float4*>(cv + j) = *reinterpret_cast<const float4*>(cs + 8 * i + j);
    *reinterpret_cast<float4*>(sv + j) = *reinterpret_cast<const float4*>(cs + n + 8 * i + j);
  }
  float y[8], w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = x[j] * cv[j] - z[j] * sv[j];
    w[j] = z[j] * cv[j] + x[j] * sv[j];
  }
  store8<T>(dst + c, y);
  store8<T>(dst + c + n, w);
}

// One block per token and slice of its pieces.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendProblem p) {
  const int t = blockIdx.x;
  const int pos = p.positions[t];
  if (pos == -1) return;  // a padding row
  const int r = p.requests ? p.requests[t] : t;
  int64_t block = -1;
  int row = 0;
  if (pos >= 0 && r >= 0 && r < p.B && pos < p.cap_rows && (!p.cos_sin || pos < p.table_rows)) {
    if (p.page_table) {
      block = p.page_table[(int64_t)r * p.pt_sb + (pos >> 6)];
      if (block < 0 || block >= p.num_blocks) block = -1;
      row = pos & 63;
    } else {
      block = r;
      row = pos;
    }
  }
  if (block < 0) {
    if (threadIdx.x == 0) atomicCAS(&g_kv_append_status, 0, TPLA_ERR_DEVICE_BOUNDS);
    return;
  }
  const float* cs = p.cos_sin ? p.cos_sin + (int64_t)pos * p.cs_s : nullptr;
  const int nk = p.k_pieces * p.Hkv, nv = p.v_pieces * p.Hkv, nq = p.q_pieces * p.Hq;
  for (int i = blockIdx.y * kThreads + threadIdx.x; i < nk + nv + nq; i += gridDim.y * kThreads) {
    if (i < nk) {
      const int h = i / p.k_pieces, j = i - h * p.k_pieces;
      row_piece<T>(p.k, t * p.k_st + h * p.k_sh, p.kv_f32,
                   reinterpret_cast<uint16_t*>(p.k_cache) + block * p.kc_s0 + row * p.kc_s1 +
                       h * p.kc_s2,
                   j, p.rot, p.k_off, p.interleaved, cs);
    } else if (i < nk + nv) {
      const int e = i - nk, h = e / p.v_pieces, j = e - h * p.v_pieces;
      row_piece<T>(p.v, t * p.v_st + h * p.v_sh, p.kv_f32,
                   reinterpret_cast<uint16_t*>(p.v_cache) + block * p.vc_s0 + row * p.vc_s1 +
                       h * p.vc_s2,
                   j, 0, 0, false, nullptr);
    } else {
      const int e = i - nk - nv, h = e / p.q_pieces, j = e - h * p.q_pieces;
      row_piece<T>(p.q, t * p.q_st + h * p.q_sh, p.q_f32,
                   reinterpret_cast<uint16_t*>(p.q_out) + t * p.qo_st + h * p.qo_sh, j, p.rot,
                   p.q_off, p.interleaved, cs);
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendProblem& p, cudaStream_t stream) {
  const int64_t pieces = (int64_t)(p.k_pieces + p.v_pieces) * p.Hkv + (int64_t)p.q_pieces * p.Hq;
  if (p.T == 0 || pieces == 0) return cudaSuccess;
  const int slices = (int)((pieces + kThreads - 1) / kThreads);
  const dim3 grid(p.T, slices < 64 ? slices : 64);
  if (p.f16)
    kv_append_kernel<F16><<<grid, kThreads, 0, stream>>>(p);
  else
    kv_append_kernel<Bf16><<<grid, kThreads, 0, stream>>>(p);
  count_launch();
  return cudaGetLastError();
}

cudaError_t status_read_clear_kv_append(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_append_status, sizeof(int));
  if (e != cudaSuccess) return e;
  if (v != 0) {
    int zero = 0;
    e = cudaMemcpyToSymbol(g_kv_append_status, &zero, sizeof(int));
  }
  *code = v;
  return e;
}

}  // namespace tpla
