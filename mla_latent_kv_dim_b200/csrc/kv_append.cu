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
// read once and written once in 16-byte pieces (8 values).  A thread owns one
// piece of the row (a plain copy, or both halves of its pairs, so that queries
// may be rotated in place) of one head, for all tokens of its block: the chain
// of position, request and page is followed once a token, by one thread, while
// the others' first values are on their way.
//
// Measured (B200, the public Python call on data that the L2 does not hold):
// sixteen prompts, 11900 tokens of 8 + 8 heads of 128 and 64 queries, f32 in and
// f16 out, 733 MB: 141 us, 5.2 TB/s, 80 % of a copy's rate; 4096 latent rows with
// the rope columns of 128 heads' queries, 144 MB: 33.5 us, 66 % (one wave of
// blocks, one token ahead, 72 of a key block's 128 threads in use); one token of
// 64 requests: 4.1 us, a launch and the chain of position, page and row.
#include <stdint.h>

#include "internal.h"
#include "kv_ptx.cuh"

namespace tpla {
namespace {

using namespace kvx;

__device__ int g_kv_append_status;

constexpr int kThreads = 128;
// Tokens of a block in a large call; 4, 8, 16, 32: 155, 144, 140, 142 us for the
// sixteen prompts above in a replayed graph (256 threads: 154)
constexpr int kTokens = 16;

// 8 consecutive values as they stand in memory: 16 or 32 bytes
template <bool F32>
struct Raw8 {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* at) {
    v[0] = reinterpret_cast<const uint4*>(at)[0];
    if (F32) v[F32 ? 1 : 0] = reinterpret_cast<const uint4*>(at)[1];
  }
  // values 4 e .. 4 e + 3
  template <typename T>
  __device__ __forceinline__ void get4(int e, float (&x)[4]) const {
    if (F32) {
      const uint4 w = v[F32 ? e : 0];
      x[0] = __uint_as_float(w.x);
      x[1] = __uint_as_float(w.y);
      x[2] = __uint_as_float(w.z);
      x[3] = __uint_as_float(w.w);
    } else {
      const float2 a = T::unpack(e ? v[0].z : v[0].x), b = T::unpack(e ? v[0].w : v[0].y);
      x[0] = a.x;
      x[1] = a.y;
      x[2] = b.x;
      x[3] = b.y;
    }
  }
  template <typename T>
  __device__ __forceinline__ uint4 to16() const {
    if (!F32) return v[0];
    float a[4], b[4];
    get4<T>(0, a);
    get4<T>(1, b);
    return make_uint4(T::pack(a[0], a[1]), T::pack(a[2], a[3]), T::pack(b[0], b[1]),
                      T::pack(b[2], b[3]));
  }
};

// What a block works on: the rows of one tensor.
struct Rows {
  const void* src;
  int64_t s_t, s_h;           // token and head strides
  uint16_t* dst;
  int64_t d0, d1, d_h;        // page (or token), row and head strides
  int heads, pieces, rot, off;
  bool by_token;              // d0 is a token stride (queries)
};

// One piece of the rows of `tn` tokens from t0 on; the next token's values are
// on their way while this one's are turned and stored.
template <typename T, bool F32, bool INTER>
__device__ __forceinline__ void do_rows(const KvAppendProblem& p, const Rows& r, int slice, int t0,
                                        int tn, const int* s_pos, const int* s_row,
                                        const long long* s_block) {
  constexpr int kE = F32 ? 4 : 2;
  const int i = slice * kThreads + threadIdx.x;
  const bool idle = i >= r.heads * r.pieces;
  const int h = idle ? 0 : i / r.pieces, j = idle ? 0 : i - h * r.pieces;
  const int n = r.rot >> 1;
  // pieces of rotated pairs come first, then plain copies
  const int pairs = INTER ? r.rot >> 3 : r.rot >> 4;
  const bool turn = j < pairs;
  int c = turn ? r.off + (j << 3) : (j - pairs) << 3;
  if (!turn && c >= r.off) c += r.rot;
  const char* src = reinterpret_cast<const char*>(r.src) + (t0 * r.s_t + h * r.s_h + c) * kE;
  uint16_t* dst = r.dst + h * r.d_h + c;
  Raw8<F32> lo, hi;
  if (!idle) {
    lo.load(src);
    if (!INTER && turn) hi.load(src + n * kE);
  }
  __syncthreads();
  if (idle) return;
  for (int u = 0; u < tn; ++u) {
    const int pos = s_pos[u];
    const Raw8<F32> a = lo, b = hi;
    src += r.s_t * kE;
    if (u + 1 < tn) {
      lo.load(src);
      if (!INTER && turn) hi.load(src + n * kE);
    }
    if (pos == -1) continue;
    uint16_t* to =
        dst + (r.by_token ? (t0 + u) * r.d0 : s_block[u] * r.d0 + s_row[u] * r.d1);
    if (!turn) {
      *reinterpret_cast<uint4*>(to) = a.template to16<T>();
      continue;
    }
    const float* cs = p.cos_sin + (int64_t)pos * p.cs_s + (INTER ? 4 * j : 8 * j);
    if (INTER) {
      const float4 co = *reinterpret_cast<const float4*>(cs);
      const float4 si = *reinterpret_cast<const float4*>(cs + n);
      float x[4], y[4];
      a.template get4<T>(0, x);
      a.template get4<T>(1, y);
      *reinterpret_cast<uint4*>(to) =
          make_uint4(T::pack(x[0] * co.x - x[1] * si.x, x[1] * co.x + x[0] * si.x),
                     T::pack(x[2] * co.y - x[3] * si.y, x[3] * co.y + x[2] * si.y),
                     T::pack(y[0] * co.z - y[1] * si.z, y[1] * co.z + y[0] * si.z),
                     T::pack(y[2] * co.w - y[3] * si.w, y[3] * co.w + y[2] * si.w));
    } else {
      uint32_t lo16[4], hi16[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 co = *reinterpret_cast<const float4*>(cs + 4 * e);
        const float4 si = *reinterpret_cast<const float4*>(cs + n + 4 * e);
        float x[4], z[4];
        a.template get4<T>(e, x);
        b.template get4<T>(e, z);
        lo16[2 * e] = T::pack(x[0] * co.x - z[0] * si.x, x[1] * co.y - z[1] * si.y);
        lo16[2 * e + 1] = T::pack(x[2] * co.z - z[2] * si.z, x[3] * co.w - z[3] * si.w);
        hi16[2 * e] = T::pack(z[0] * co.x + x[0] * si.x, z[1] * co.y + x[1] * si.y);
        hi16[2 * e + 1] = T::pack(z[2] * co.z + x[2] * si.z, z[3] * co.w + x[3] * si.w);
      }
      *reinterpret_cast<uint4*>(to) = make_uint4(lo16[0], lo16[1], lo16[2], lo16[3]);
      *reinterpret_cast<uint4*>(to + n) = make_uint4(hi16[0], hi16[1], hi16[2], hi16[3]);
    }
  }
}

// TB: tokens of a block.  blockIdx.y: slices of kThreads pieces, those of the
// keys first, then the values', then the queries'.
template <typename T, int TB, bool KVF32, bool QF32, bool INTER>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendProblem p) {
  __shared__ int s_pos[TB];  // -1: nothing to do
  __shared__ int s_row[TB];
  __shared__ long long s_block[TB];
  const int t0 = blockIdx.x * TB, tn = min(TB, p.T - t0);
  if (threadIdx.x < tn) {
    const int t = t0 + threadIdx.x;
    int pos = p.positions[t], row = 0;
    long long block = 0;
    if (pos != -1) {  // not a padding row
      const int req = p.requests ? p.requests[t] : t;
      bool ok = pos >= 0 && req >= 0 && req < p.B && pos < p.cap_rows &&
                (!p.cos_sin || pos < p.table_rows);
      if (ok) {
        block = req;
        row = pos;
        if (p.page_table) {
          block = p.page_table[(int64_t)req * p.pt_sb + (pos >> 6)];
          row = pos & 63;
          ok = block >= 0 && block < p.num_blocks;
        }
      }
      if (!ok) {
        atomicCAS(&g_kv_append_status, 0, TPLA_ERR_DEVICE_BOUNDS);
        pos = -1;
      }
    }
    s_pos[threadIdx.x] = pos;
    s_row[threadIdx.x] = row;
    s_block[threadIdx.x] = block;
  }
  const int ks = (p.k_pieces * p.Hkv + kThreads - 1) / kThreads;
  const int vs = (p.v_pieces * p.Hkv + kThreads - 1) / kThreads;
  const int y = blockIdx.y;
  if (y < ks) {
    const Rows r = {p.k, p.k_st, p.k_sh, reinterpret_cast<uint16_t*>(p.k_cache), p.kc_s0, p.kc_s1,
                    p.kc_s2, p.Hkv, p.k_pieces, p.rot, p.k_off, false};
    do_rows<T, KVF32, INTER>(p, r, y, t0, tn, s_pos, s_row, s_block);
  } else if (y < ks + vs) {
    const Rows r = {p.v, p.v_st, p.v_sh, reinterpret_cast<uint16_t*>(p.v_cache), p.vc_s0, p.vc_s1,
                    p.vc_s2, p.Hkv, p.v_pieces, 0, 0, false};
    do_rows<T, KVF32, true>(p, r, y - ks, t0, tn, s_pos, s_row, s_block);
  } else {
    const Rows r = {p.q, p.q_st, p.q_sh, reinterpret_cast<uint16_t*>(p.q_out), p.qo_st, 0,
                    p.qo_sh, p.Hq, p.q_pieces, p.rot, p.q_off, true};
    do_rows<T, QF32, INTER>(p, r, y - ks - vs, t0, tn, s_pos, s_row, s_block);
  }
}

template <typename T, bool KVF32, bool QF32, bool INTER>
void launch_form(const KvAppendProblem& p, int slices, cudaStream_t stream) {
  // Many tokens a block once that still gives every SM the blocks it can hold,
  // else one: the latency counts.
  if ((int64_t)p.T * slices >= (int64_t)sm_count(current_device()) * 8 * kTokens)
    kv_append_kernel<T, kTokens, KVF32, QF32, INTER>
        <<<dim3((p.T + kTokens - 1) / kTokens, slices), kThreads, 0, stream>>>(p);
  else
    kv_append_kernel<T, 1, KVF32, QF32, INTER>
        <<<dim3(p.T, slices), kThreads, 0, stream>>>(p);
}

template <typename T, bool KVF32, bool QF32>
void launch_style(const KvAppendProblem& p, int slices, cudaStream_t stream) {
  if (p.interleaved)
    launch_form<T, KVF32, QF32, true>(p, slices, stream);
  else
    launch_form<T, KVF32, QF32, false>(p, slices, stream);
}

template <typename T>
void launch_type(const KvAppendProblem& p, int slices, cudaStream_t stream) {
  if (p.kv_f32)
    p.q_f32 ? launch_style<T, true, true>(p, slices, stream)
            : launch_style<T, true, false>(p, slices, stream);
  else
    p.q_f32 ? launch_style<T, false, true>(p, slices, stream)
            : launch_style<T, false, false>(p, slices, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendProblem& p, cudaStream_t stream) {
  auto slices_of = [](int64_t pieces) { return (int)((pieces + kThreads - 1) / kThreads); };
  const int slices = slices_of((int64_t)p.k_pieces * p.Hkv) +
                     slices_of((int64_t)p.v_pieces * p.Hkv) +
                     slices_of((int64_t)p.q_pieces * p.Hq);
  if (p.T == 0 || slices == 0) return cudaSuccess;
  if (slices > 65535) return cudaErrorInvalidValue;
  if (p.f16)
    launch_type<F16>(p, slices, stream);
  else
    launch_type<Bf16>(p, slices, stream);
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
