// Causal (or full) attention of packed prompts over uncompressed keys and
// values, with grouped heads, on the 5th-generation tensor cores:
//   s_ij = scale q_i . k_j,  j < limit_i;   out_i = sum_j softmax(s_i)_j v_j,
//   lse_i = ln sum_j exp(s_ij);   limit_i = L or, causal, L - T + i + 1
// for a request's T new tokens against its L keys (packed rows, or the paged
// cache with the prompt's own keys already in it).
//
// The two matrix products bound it (2 (Dk + Dv) flops a pair and head), and
// beside them the exponentials: one per score on a unit that gives 16 a cycle
// against the 128 x 128 x 16 product's 64 cycles.  So:
//  * a tile is 128 rows: tpt = 128 / g tokens times the g query heads of one
//    key head (row = token * g + head), so that grouped heads share every
//    key and value tile and few tokens still fill the rows;
//  * a work item is two such tiles A and B of consecutive tokens, which share
//    the key tiles of 64 keys.  Each has a softmax warpgroup, O in TMEM and
//    two S buffers of 64 columns there: while the softmax works on one S the
//    tensor core fills the other, so neither waits out the other's latency.
//    Three threads issue the products (Q K^T of A, of B, and both P V), so
//    that the waits of one pass while the others feed the tensor core.  P goes
//    over its own S as 16-bit pairs, the A operand from TMEM: 2 x (128 + Dv)
//    of the 512 columns in all.  (With one S of 128 keys a tile Q K^T waits for
//    P V, P V for the softmax and the softmax for Q K^T: 4450 cycles for 128
//    keys of both tiles against 2048 of tensor work.  In exchange N = 64 takes
//    48 cycles where N = 128 takes 64, because Q is read again: 1152 cycles for
//    64 keys of both tiles at 128 columns);
//  * a thread owns a row: no exchange for the row maximum.  O is rescaled
//    only when the maximum has grown by more than 2^8 (fp16: 2^6);
//  * K and V tiles go through a ring of key tiles (64-column chunks of 64 rows,
//    128-byte swizzle, K-major for Q K^T and MN-major for P V);
//  * items are handed out longest first (a small kernel sorts them; one
//    request needs no sorting), so the last ones are short.  Where a call has
//    too few items for the GPU (a short chunk after a long prefix), that
//    kernel cuts their keys into pieces, whose normalised results a third
//    kernel joins by their log-sum-exp.
//
// Measured (B200, the public Python call on data that the L2 does not hold, bf16
// in and out; of the burst rate of a library product, 1651 TFLOP/s): 16384 tokens
// of 8 heads over one of 128: 527 us, 1040 TFLOP/s, 63 %; 128 heads of 4096
// tokens, 192 / 128 wide: 752 us, 55 %; chunks of four prompts after 4000 to 8000
// tokens (f16, paged): 208 us, 48 %; twelve prompts of 33 to 1500 tokens: 96 us,
// 35 %; one of 77 tokens: 9.4 us, mostly fixed (an empty kernel takes 1 us, the
// start 2, a chain of two key tiles 3).  Replayed graphs, which find their data
// in the L2 and were taken at 1.97 GHz, take 451, 648, 177, 86 and 7.6 us.
//
// What bounds it is feeding the tensor core: of 1750 cycles a step of 64 keys at
// Dk = 128 its pipe is taken 82 % of the time (1430 cycles, 1024 of them at the
// full rate), the exponential unit 44 %, the schedulers 53 %; beyond that the two
// warpgroups reach the exponentials at the same time.  (Two warpgroups a query
// tile, 16 softmax warps of 104 registers, in three forms: 8 to 25 % slower.)
// The short calls end in blocks with nothing left to do.
#include <cuda_runtime.h>

#include <mutex>

#include "internal.h"
#include "kv_map.h"
#include "kv_ptx.cuh"

namespace tpla {
namespace {

using namespace kvx;

__device__ int g_kv_prefill_status;

constexpr int kRows = 128;    // rows of a query tile
constexpr int kKeys = 64;     // keys of a key tile
constexpr int kChunk = 8192;  // 64 keys x 64 columns
constexpr int kThreads = 384;
// Warps 0 and 1 load the query tiles A and B and issue their Q K^T, 2 issues
// P V of both, 3 loads key tiles; 4-7 and 8-11 are the softmax warpgroups of A
// and B.
constexpr int kWarpQK = 0, kWarpPV = 2, kWarpProd = 3, kWarpSm0 = 4;
constexpr int kMaxRing = 12;   // key tiles
constexpr int kFlagRing = 16;  // key tiles whose page flags are kept (> kMaxRing + 2)
constexpr int kSmemBytes = 232448;
constexpr int kMiscBytes = 2048;
constexpr int kBuckets = 2048;  // of the items' lengths
constexpr uint32_t kColS = 0, kColO = 256;

// One pair of weights in this many comes from the FMA pipe instead of the
// exponential unit, which both warpgroups wait for at the same time.  None, one
// in 8, 4, 3, replayed: chunk of four prompts 200, 194, 184, 185 us; packed 91,
// 87, 84, 85.  Not where Dk is 192: there Q K^T takes longer than the exponentials
// (128 heads of 4096 tokens, replayed: 695 us without, 708 with).
constexpr int kFmaEvery = 4;
constexpr int64_t kL2Share = 96 << 20;  // bytes of keys and values that the L2 keeps
constexpr int kMinPiece = 8;  // key tiles; a shorter piece is mostly fixed work

struct alignas(16) Entry {  // two query tiles of one request; moved as three int4
  int t0;       // first token within the request
  int q0, qlen; // the request's rows of q
  int k0;       // packed: its first row of k
  int kvlen;    // its keys
  int b;
  int j0, j1;   // key tiles of this piece
  int slot;     // of its partial result (times the heads), -1: the whole item
  int pad[3];
};
static_assert(sizeof(Entry) == 48 && alignof(Entry) == 16, "three int4");

struct Join {  // an item in pieces
  int t0, q0, qlen, slot, pieces, pad[3];
};

struct Params {
  const int *cu_q, *cu_k, *seq_lens, *page_table;
  int64_t pt_sb;
  int num_blocks;
  int cap_rows;
  int B, T, Hkv, g, gg, groups, tpt;  // gg heads of a row group, tpt tokens of a tile
  int paired;            // the order of the items, see Items
  int causal;
  float scale_log2;      // |softmax scale| * log2(e), > 0 (see the launcher)
  int negate;            // scale < 0
  const int* count;      // entries of the list (and of joins), or null: one request, no list
  const Entry* list;
  const Join* joins;
  float* part_o;         // [slot * heads + head, Dv / 4, rows_slot, 4]
  float* part_l;         // [slot * heads + head, rows_slot]
  int rows_slot;         // 2 tpt gg, less where the call has fewer tokens
  void* out;
  int out_dtype;
  int out32;             // 16-bit rows on 32-byte boundaries
  int64_t o_st, o_sh;
  float* lse;
  int64_t l_st, l_sh;
};

struct Item {
  Entry e;
  int hk, rg;
  int slot;
  int n[2];  // key tiles of the two query tiles in this piece
  int nmax;
};

__device__ __forceinline__ void bounds() {
  atomicCAS(&g_kv_prefill_status, 0, TPLA_ERR_DEVICE_BOUNDS);
}

// A request's rows of q and keys, clipped to the tensors.
__device__ __forceinline__ void request(const Params& p, int b, Entry& e) {
  const int a = p.cu_q[b], z = p.cu_q[b + 1];
  const int lo = max(0, min(a, p.T)), hi = max(lo, min(z, p.T));
  bool bad = lo != a || hi != z;
  e.b = b;
  e.q0 = lo;
  e.qlen = hi - lo;
  if (p.page_table) {
    const int n = p.seq_lens[b];
    e.k0 = 0;
    e.kvlen = max(0, min(n, p.cap_rows));
    bad |= e.kvlen != n;
  } else {
    const int ka = p.cu_k[b], kz = p.cu_k[b + 1];
    const int kl = max(0, min(ka, p.cap_rows)), kh = max(kl, min(kz, p.cap_rows));
    bad |= kl != ka || kh != kz;
    e.k0 = kl;
    e.kvlen = kh - kl;
  }
  if (bad) bounds();
}

// Keys that token `tok` of the request sees.
__device__ __forceinline__ int limit_of(const Params& p, const Entry& e, int tok) {
  if (!p.causal) return e.kvlen;
  return max(0, min(e.kvlen, e.kvlen - e.qlen + tok + 1));
}

__device__ __forceinline__ int item_count(const Params& p) {
  int n;
  if (p.count) {
    n = *p.count;
  } else {
    Entry e;
    request(p, 0, e);
    n = (e.qlen + 2 * p.tpt - 1) / (2 * p.tpt);
  }
  return n * p.Hkv * p.groups;
}

// A block's items: every gridDim.x-th of the list, in alternating direction
// so that the blocks with the longest of one round get the shortest of the
// next.  Or (`paired`: one prompt) head after head, a long item and the short
// one that makes up for it together, so that every pair is the same work and
// few heads' keys and values are in use at a time.
struct Items {
  int total, heads, round;
  __device__ explicit Items(const Params& p)
      : total(item_count(p)), heads(p.Hkv * p.groups), round(0) {}

  // the next item with keys, or (want_empty) the next of any kind
  __device__ bool next(const Params& p, Item& it, bool want_empty = false) {
    for (;;) {
      int x, h;
      if (p.paired) {
        const int entries = total / heads, pairs = (entries + 1) / 2;
        const long long at = (long long)(round >> 1) * gridDim.x, pair = at + blockIdx.x;
        const bool second = round & 1;
        if (at >= (long long)pairs * heads) return false;
        ++round;
        if (pair >= (long long)pairs * heads) continue;
        h = (int)pair / pairs;
        x = (int)pair - h * pairs;
        if (second) {
          if (x == entries - 1 - x) continue;  // the middle one has no other
          x = entries - 1 - x;
        }
      } else {
        const int c = round & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
        const long long idx = (long long)round * gridDim.x + c;
        if ((long long)round * gridDim.x >= total) return false;
        ++round;
        if (idx >= total) continue;
        x = (int)idx / heads;
        h = (int)idx - x * heads;
      }
      get(p, x, h, it);
      if (it.nmax > 0 || want_empty) return true;
    }
  }

  __device__ void get(const Params& p, int x, int h, Item& it) const {
    it.hk = h / p.groups;
    it.rg = h - it.hk * p.groups;
    if (p.count) {
      const int4* s = reinterpret_cast<const int4*>(p.list + x);
      int4* d = reinterpret_cast<int4*>(&it.e);
      d[0] = s[0];
      d[1] = s[1];
      d[2] = s[2];
    } else {  // longest first: the last tokens of a causal prompt see the most keys
      request(p, 0, it.e);
      it.e.t0 = (total / heads - 1 - x) * 2 * p.tpt;
      it.e.j0 = 0;
      it.e.j1 = 1 << 30;
      it.e.slot = -1;
    }
    it.slot = it.e.slot < 0 ? -1 : it.e.slot * heads + h;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int a = it.e.t0 + t * p.tpt, z = min(a + p.tpt, it.e.qlen);
      const int n = z > a ? (limit_of(p, it.e, z - 1) + kKeys - 1) / kKeys : 0;
      it.n[t] = max(0, min(n, it.e.j1) - it.e.j0);
    }
    it.nmax = max(it.n[0], it.n[1]);
    // A query tile that sees no key, or has no rows, takes part with all its
    // scores masked or unused: so the two tiles are never more than two key
    // tiles apart (128 tokens), and no barrier is waited for from two phases
    // away, where its parity would say the wrong thing.
    if (it.n[0] == 0) it.n[0] = it.nmax;
    if (it.n[1] == 0) it.n[1] = it.nmax;
  }
};

template <typename T, int DK, int DV>
struct Cfg {
  static constexpr int kNK = DK / 64, kNV = DV / 64;  // 64-column chunks
  static constexpr int kQTile = kNK * kRows * 128;    // bytes of a query tile
  static constexpr int kKV = (kNK + kNV) * kChunk;    // bytes of a key tile
  static constexpr int kRing0 = (kSmemBytes - 1024 - kMiscBytes - 2 * kQTile) / kKV;
  static constexpr int kRing = kRing0 < kMaxRing ? kRing0 : kMaxRing;
  static constexpr int kSmem = 1024 + 2 * kQTile + kRing * kKV + kMiscBytes;
  // Q K^T runs up to two key tiles ahead of P V
  static_assert(kSmem <= kSmemBytes && kRing >= 3, "shared memory");
  static constexpr uint32_t idesc(int n, bool b_mn) {
    return (1u << 4) | ((uint32_t)T::kFormat << 7) | ((uint32_t)T::kFormat << 10) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
  }
};

struct Misc {
  // per ring slot: K and V landed; K no longer needed by either softmax
  // (their S are made), V no longer by P V
  unsigned long long full[kMaxRing][2], empty[kMaxRing][2];
  unsigned long long q_full[2], q_empty[2];
  // per query tile and S buffer: S made, P stored, P V done
  unsigned long long s_full[2][2], p_full[2][2], pv_done[2][2];
  int flags[kFlagRing];
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc shared memory");

// Key tiles: a chunk from a lane of its own, because a thread's copies land
// one after another.
template <typename T, int DK, int DV>
__device__ void producer(const Params& p, const CUtensorMap* km, const CUtensorMap* vm,
                         uint32_t sbase, Misc& ms) {
  using C = Cfg<T, DK, DV>;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &ms.abort_flag;
  Items items(p);
  Item it;
  uint32_t slot = 0, phase = 1;
  uint32_t tile = 0, sent[2] = {0, 0};  // K and V tiles under way or landed
  int ok = 1;
  while (ok && items.next(p, it)) {
    int win = 0;  // lane i: the page id of key tile 32 w + i
    for (int j = 0; ok && j < it.nmax; ++j, ++tile) {
      int page = 0, row = it.e.k0 + kKeys * (it.e.j0 + j), flag = 0;
      if (p.page_table) {
        if ((j & 31) == 0)
          win = j + lane < it.nmax
                    ? p.page_table[(int64_t)it.e.b * p.pt_sb + it.e.j0 + j + lane]
                    : 0;
        page = __shfl_sync(0xffffffffu, win, j & 31);
        row = 0;
        if (page < 0 || page >= p.num_blocks) {
          flag = 1;
          page = max(p.num_blocks, 1);  // past the last page: reads as zeros
        }
      }
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        constexpr int kN[2] = {C::kNK, C::kNV};
        const uint32_t full = smem_addr(&ms.full[slot][v]);
        if (lane == 0) {
          if (tile >= C::kRing)
            ok = wait_bar(smem_addr(&ms.empty[slot][v]), phase, abort_flag, &g_kv_prefill_status);
          if (ok) {
            if (v == 0) {
              if (flag) bounds();
              ms.flags[tile % kFlagRing] = flag;
            }
            mbar_arrive_expect_tx(full, kN[v] * kChunk);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        sent[v] = tile + 1;
        const int c = lane - (v ? C::kNK : 0);
        if (c >= 0 && c < kN[v])
          tma_load_5d(sbase + 2 * C::kQTile + slot * C::kKV + lane * kChunk, v ? vm : km, 0, row, c,
                      it.hk, page, full);
      }
      if (++slot == C::kRing) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  if (lane < 2) {  // no copy outlives the block, whatever the other roles do
    const long long since = clock64();
    const uint32_t n = lane ? sent[1] : sent[0];
    for (uint32_t i = n < C::kRing ? 0 : n - C::kRing; i < n; ++i)
      wait_landed(smem_addr(&ms.full[i % C::kRing][lane]), (i / C::kRing) & 1, since);
  }
}

// Query tile t: its loads, and S = Q K^T of each key tile into the S buffer
// whose P V is done, two key tiles ahead of P V.
template <typename T, int DK, int DV>
__device__ void qk_issuer(const Params& p, const int t, const CUtensorMap* qm, uint32_t sbase,
                          uint32_t tmem, Misc& ms) {
  using C = Cfg<T, DK, DV>;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &ms.abort_flag;
  const uint64_t dQ = sw128_desc(sbase + t * C::kQTile, 16, 1024);
  const uint64_t dK = sw128_desc(sbase + 2 * C::kQTile, 16, 1024);
  constexpr uint32_t kC = kChunk >> 4, kT = C::kKV >> 4;
  const uint32_t q_lo = (uint32_t)dQ, k_lo = (uint32_t)dK, hi = (uint32_t)(dK >> 32);
  const uint32_t tS = tmem + kColS + kRows * t;
  // a negative scale: bit 13 negates A, so that the maximum is still a maximum
  const uint32_t idesc = C::idesc(kKeys, false) | (p.negate ? 1u << 13 : 0u);
  const uint32_t q_full = smem_addr(&ms.q_full[t]), q_empty = smem_addr(&ms.q_empty[t]);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return wait_bar(bar, parity, abort_flag, &g_kv_prefill_status);
  };
  Items items(p);
  Item it;
  uint32_t cnt = 0, slot = 0, phase = 0;
  for (uint32_t i = 0; items.next(p, it); ++i) {
    const int n = t ? it.n[1] : it.n[0];
    int ok = 1;
    if (lane == 0) {
      ok = i == 0 || wait(q_empty, (i - 1) & 1);
      if (ok) mbar_arrive_expect_tx(q_full, C::kNK * p.gg * p.tpt * 128);
    }
    if (!__shfl_sync(0xffffffffu, ok, 0)) return;
    if (lane < C::kNK)  // a thread's copies land one after another
      tma_load_5d(sbase + t * C::kQTile + lane * kRows * 128, qm, 0, it.rg * p.gg,
                  it.e.q0 + it.e.t0 + t * p.tpt, lane, it.hk, q_full);
    __syncwarp();
    if (lane == 0) {
      ok = wait(q_full, i & 1);
      if (!ok) wait_landed(q_full, i & 1, clock64());
      for (int j = 0; ok && j < n; ++j, ++cnt) {
        const uint32_t buf = cnt & 1;
        ok = wait(smem_addr(&ms.full[slot][0]), phase) &&
             (cnt < 2 || wait(smem_addr(&ms.pv_done[t][buf]), ((cnt - 2) >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t k0 = k_lo + slot * kT, dS = tS + kKeys * buf;
#pragma unroll
        for (int c = 0; c < C::kNK; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(dS, q_lo + 2 * c * kC + 2 * k, hi, k0 + c * kC + 2 * k, hi,
                   idesc, (c | k) != 0);
        commit(smem_addr(&ms.s_full[t][buf]));
        if (++slot == C::kRing) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (ok) commit(q_empty);
    }
    if (!__shfl_sync(0xffffffffu, ok, 0)) return;
    slot = __shfl_sync(0xffffffffu, slot, 0) + (it.nmax - n);  // the other query tile's
    phase = __shfl_sync(0xffffffffu, phase, 0);
    if (slot >= C::kRing) {
      slot -= C::kRing;
      phase ^= 1;
    }
    cnt = __shfl_sync(0xffffffffu, cnt, 0);
  }
}

// O += P V of both query tiles, key tile by key tile.
template <typename T, int DK, int DV>
__device__ void pv_issuer(const Params& p, uint32_t sbase, uint32_t tmem, Misc& ms) {
  using C = Cfg<T, DK, DV>;
  volatile int* abort_flag = &ms.abort_flag;
  // V, MN-major: rows are keys, 64 columns to a 128-byte row, column groups a
  // chunk apart
  const uint64_t dV = sw128_desc(sbase + 2 * C::kQTile + C::kNK * kChunk, kChunk, 1024);
  constexpr uint32_t kT = C::kKV >> 4;
  const uint32_t v_lo = (uint32_t)dV, v_hi = (uint32_t)(dV >> 32);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return wait_bar(bar, parity, abort_flag, &g_kv_prefill_status);
  };
  Items items(p);
  Item it;
  uint32_t cnt[2] = {0, 0}, slot = 0, phase = 0;
  while (items.next(p, it)) {
    for (int j = 0; j < it.nmax; ++j) {
      if (!wait(smem_addr(&ms.full[slot][1]), phase)) return;
      const uint32_t v0 = v_lo + slot * kT;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (j >= it.n[t]) continue;
        const uint32_t buf = cnt[t] & 1;
        if (!wait(smem_addr(&ms.p_full[t][buf]), (cnt[t] >> 1) & 1)) return;
        ++cnt[t];
        tc_fence_after();
        const uint32_t pS = tmem + kColS + kRows * t + kKeys * buf, tO = tmem + kColO + 128 * t;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts(tO, pS + 8 * k, v0 + 128 * k, v_hi, C::idesc(DV, true), (j | k) != 0);
        commit(smem_addr(&ms.pv_done[t][buf]));
      }
      commit(smem_addr(&ms.empty[slot][1]));
      if (++slot == C::kRing) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
}

template <typename T, int DK, int DV>
__device__ void softmax(const Params& p, const int t, uint32_t sbase, uint32_t tmem, Misc& ms) {
  using C = Cfg<T, DK, DV>;
  volatile int* abort_flag = &ms.abort_flag;
  const int w = (int)(threadIdx.x >> 5) & 3;
  const int row = 32 * w + (int)(threadIdx.x & 31);  // this thread's row and TMEM lane
  const uint32_t lane_base = (uint32_t)(32 * w) << 16;
  const uint32_t tS = tmem + lane_base + kColS + kRows * t;
  const uint32_t tO = tmem + lane_base + kColO + 128 * t;
  const int my_tok = row / p.gg, my_head = row - my_tok * p.gg;
  uint32_t cnt = 0, tiles = 0;
  const bool leader = (threadIdx.x & 127) == 0;
  // this query tile needs the key tile's K no longer; the other says so too
  auto release = [&](uint32_t tile) {
    if (leader) arrive(smem_addr(&ms.empty[tile % C::kRing][0]));
  };
  auto wait = [&](unsigned long long& bar, uint32_t parity) {
    const bool ok = wait_bar(smem_addr(&bar), parity, abort_flag, &g_kv_prefill_status);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  Items items(p);
  Item it;
  while (items.next(p, it, true)) {
    const int tok = it.e.t0 + t * p.tpt + my_tok;
    const int head = it.rg * p.gg + my_head;
    const bool live = my_tok < p.tpt && tok < it.e.qlen && head < p.g;
    // rows past the tile's tokens or the request's are computed and not stored
    const int held = it.e.kvlen - kKeys * it.e.j0;  // keys from this piece's first on
    const int limit = (live ? limit_of(p, it.e, tok) : it.e.kvlen) - kKeys * it.e.j0;
    const int n = t ? it.n[1] : it.n[0];
    // The maximum, and the f32 sum of the weights before their rounding to 16
    // bits for P V: only the numerator carries that rounding (half a step a
    // weight).  Summing the rounded weights too, as the divisor, took 3-4 % of
    // the time and gained 2 % of the error (mean relative 2.10e-3 / 2.14e-3).
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j, ++cnt) {
      const int buf = cnt & 1;
      const uint32_t ts = tS + kKeys * buf;
      if (!wait(ms.s_full[t][buf], (cnt >> 1) & 1)) return;
      tc_fence_after();
      release(tiles + j);
      int nv = limit - kKeys * j;
      if (p.page_table && ms.flags[(tiles + j) % kFlagRing]) nv = 0;  // a bad page
      if (__any_sync(0xffffffffu, nv < kKeys)) {
        // few key tiles: masked in place, so that the others pay only the branch
#pragma unroll 1
        for (int c = 0; c < kKeys; c += 32) {
          uint32_t r[32];
          tmem_ld32(ts + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) r[k] = c + k < nv ? r[k] : 0xff800000u;  // -inf
          tmem_st32(ts + c, r);
        }
        tmem_wait_st();
      }
      float x[kKeys];
      {
        uint32_t r[2][32];
        tmem_ld32(ts, r[0]);
        tmem_ld32(ts + 32, r[1]);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < kKeys; ++k) x[k] = __uint_as_float(r[k >> 5][k & 31]);
      }
      float mxs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mxs[i] = fmaxf(x[2 * i], x[2 * i + 1]);
#pragma unroll
        for (int k = 8 + 2 * i; k < kKeys; k += 8) mxs[i] = max3(mxs[i], x[k], x[k + 1]);
      }
      const float mx = fmaxf(max3(mxs[0], mxs[1], mxs[2]), mxs[3]) * p.scale_log2;
      const bool resc = mx > m + T::kLag && m != -INFINITY;
      if (m == -INFINITY) m = mx;
      if (__any_sync(0xffffffffu, resc)) {
        // O as the P V before this one leaves it (no maximum before the first)
        if (!wait(ms.pv_done[t][buf ^ 1], ((cnt - 1) >> 1) & 1)) return;
        tc_fence_after();
        const float factor = resc ? ex2(m - mx) : 1.f;
        if (resc) m = mx;
        l *= factor;
#pragma unroll
        for (int c = 0; c < DV; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * factor);
          tmem_st32(tO + c, o);
        }
        tmem_wait_st();
      }
      const int left = held - kKeys * j;
      if (left < kKeys) {
        // behind the request's last key stand other rows or stale ones; a
        // weight of 0 does not stop an infinity or a NaN there, so they are
        // cleared before P V reads them
        const uint32_t tile = tiles + j, slot = tile % C::kRing;
        if (!wait(ms.full[slot][1], (tile / C::kRing) & 1)) return;
        if (row >= left && row < kKeys) {
          const uint32_t v = sbase + 2 * C::kQTile + slot * C::kKV + C::kNK * kChunk + row * 128;
#pragma unroll
          for (int i = 0; i < 8 * C::kNV; ++i)
            st_shared_v4(v + (i >> 3) * kChunk + 16 * (i & 7), 0, 0, 0, 0);
        }
        fence_async_smem();
      }
      const float mu = m == -INFINITY ? 0.f : m - T::kLiftLag;
      const uint64_t sc = f2_pack(p.scale_log2, p.scale_log2), nm = f2_pack(-mu, -mu);
      uint64_t sum = f2_pack(0.f, 0.f);
      uint32_t pk[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        float e0, e1;
        const uint64_t y = f2_fma(f2_pack(x[2 * k], x[2 * k + 1]), sc, nm);
        if (DK < 192 && k % kFmaEvery == kFmaEvery / 2) {
          f2_ex2_fma(y, e0, e1);
        } else {
          f2_unpack(y, e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
        }
        pk[k] = T::pack(e0, e1);
        sum = f2_add(sum, f2_pack(e0, e1));
      }
      tmem_st32(ts, pk);  // over this row's own scores: they are in registers
      float a, b;
      f2_unpack(sum, a, b);
      l += a + b;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) arrive(smem_addr(&ms.p_full[t][buf]));
    }
    if (n > 0) {
      if (!wait(ms.pv_done[t][(cnt - 1) & 1], ((cnt - 1) >> 1) & 1)) return;
      tc_fence_after();
    }
    if (leader) {  // key tiles that only the other query tile reads, as they come
      for (int j = n; j < it.nmax; ++j) {
        const uint32_t tile = tiles + j;
        if (wait_bar(smem_addr(&ms.full[tile % C::kRing][0]), (tile / C::kRing) & 1, abort_flag,
                     &g_kv_prefill_status))
          release(tile);
      }
    }
    __syncwarp();
    tiles += it.nmax;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : NAN);
    // the row's place: in the output, or (f32) in the piece's slot
    const int64_t orow = (int64_t)(it.e.q0 + tok) * p.o_st + (int64_t)(it.hk * p.g + head) * p.o_sh;
    const int64_t prow =
        (int64_t)it.slot * p.rows_slot + (t * p.tpt + my_tok) * p.gg + my_head;
    const int prows = p.rows_slot;
    float* const part = p.part_o + ((int64_t)it.slot * (DV / 4) * prows + (t * p.tpt + my_tok) * p.gg +
                                    my_head) * 4;
    float* const frow = reinterpret_cast<float*>(p.out) + orow;
    uint16_t* const hrow = reinterpret_cast<uint16_t*>(p.out) + orow;
#pragma unroll
    for (int c = 0; c < DV; c += 32) {
      uint32_t o[32];
      if (n > 0) {
        tmem_ld32(tO + c, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
      }
      if (live) {
        if (it.slot >= 0) {  // the rows of a warp lie side by side
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<float4*>(part + (int64_t)((c + k) / 4) * prows * 4) = make_float4(
                __uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv,
                __uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv);
        } else if (p.out_dtype == TPLA_F32) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<float4*>(frow + c + k) = make_float4(
                __uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv,
                __uint_as_float(o[k + 2]) * inv, __uint_as_float(o[k + 3]) * inv);
        } else {
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[k] = T::pack(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          if (p.out32) {  // a thread's stores lie in lines of their own: the fewer the better
            st_global_v8(hrow + c, v);
            st_global_v8(hrow + c + 16, v + 8);
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<uint4*>(hrow + c + 2 * k) =
                  make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
        }
      }
    }
    if (live && (p.lse || it.slot >= 0)) {
      const float lse = l > 0.f ? (m + (log2f(l) - T::kLiftLag)) * kLn2 : (l == 0.f ? -INFINITY : NAN);
      if (it.slot >= 0)
        p.part_l[prow] = lse;
      else
        p.lse[(int64_t)(it.e.q0 + tok) * p.l_st + (int64_t)(it.hk * p.g + head) * p.l_sh] = lse;
    }
    tc_fence_before();
  }
}

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
kv_prefill_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                  const __grid_constant__ CUtensorMap vm, const Params p) {
  using C = Cfg<T, DK, DV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  Misc& ms = *reinterpret_cast<Misc*>(smem + 2 * C::kQTile + C::kRing * C::kKV);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int s = 0; s < C::kRing; ++s) {
        mbar_init(smem_addr(&ms.full[s][i]), 1);
        mbar_init(smem_addr(&ms.empty[s][i]), i == 0 ? 2 : 1);
      }
      mbar_init(smem_addr(&ms.q_full[i]), 1);
      mbar_init(smem_addr(&ms.q_empty[i]), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&ms.s_full[i][b]), 1);
        mbar_init(smem_addr(&ms.p_full[i][b]), 4);
        mbar_init(smem_addr(&ms.pv_done[i][b]), 1);
      }
    }
    ms.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpProd && lane == 0) {
    tma_prefetch(&qm);
    tma_prefetch(&km);
    tma_prefetch(&vm);
  }
  if (warp == kWarpPV) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&ms.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&ms.tmem);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the list of items

  if (warp >= kWarpSm0) {
    softmax<T, DK, DV>(p, (warp - kWarpSm0) >> 2, sbase, tmem, ms);
  } else if (warp == kWarpProd) {
    producer<T, DK, DV>(p, &km, &vm, sbase, ms);
  } else if (warp == kWarpPV) {
    if (lane == 0) pv_issuer<T, DK, DV>(p, sbase, tmem, ms);
  } else {
    qk_issuer<T, DK, DV>(p, warp - kWarpQK, &qm, sbase, tmem, ms);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpPV) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// The list of items, longest first: a counting sort by the key tiles of each
// item's last token.  One block; a warp takes a request at a time.  The order
// within a bucket is not fixed, and no result depends on it.
//
// With `cut` items may be cut: the work of a call with few items is meant to
// fill `fill` blocks twice, so no piece is longer than that share.
//
// Offsets that rise give at most `room` items, T / tb + B.  Offsets that fall
// can claim rows again and again; where they claim more items than that, the
// call is answered with no row at all, before anything is counted in 32 bits.
// With at most `room` items the list has an entry, and the pieces a slot, for
// all: with W key tiles in all items, a piece may be W heads / (2 fill) long or
// longer, so the pieces are at most W / longest <= 2 fill / heads and one an
// item; an item that is cut is longer than one piece, so there are at most
// 2 fill / heads of those and 4 fill / heads pieces of theirs.
__global__ void __launch_bounds__(1024) kv_prefill_plan_kernel(const Params p, Entry* list,
                                                               Join* joins, int* count, int room,
                                                               bool cut, int fill) {
  __shared__ int hist[kBuckets];
  __shared__ int top, warp_sum[32], n_joins, n_slots;
  __shared__ unsigned long long claimed, work;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tb = 2 * p.tpt;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < kBuckets; i += 1024) hist[i] = 0;
  if (threadIdx.x == 0) {
    top = n_joins = n_slots = 0;
    claimed = work = 0;
  }
  __syncthreads();
  auto tiles_of = [&](const Entry& e, int t0) {
    return (limit_of(p, e, min(t0 + tb, e.qlen) - 1) + kKeys - 1) / kKeys;
  };
  int most = 0;
  unsigned long long items = 0;
  for (int b = threadIdx.x; b < p.B; b += 1024) {
    Entry e;
    request(p, b, e);
    most = max(most, (e.kvlen + kKeys - 1) / kKeys);
    items += (e.qlen + tb - 1) / tb;
  }
  if (most) atomicMax(&top, most);
#pragma unroll
  for (int o = 16; o; o >>= 1) items += __shfl_down_sync(0xffffffffu, items, o);
  if (lane == 0 && items) atomicAdd(&claimed, items);
  __syncthreads();
  if (claimed > (unsigned long long)room) {
    if (threadIdx.x == 0) {
      bounds();
      count[0] = count[1] = 0;
    }
    return;
  }
  if (cut) {
    unsigned long long mine = 0;
    for (int b = warp; b < p.B; b += 32) {
      Entry e;
      request(p, b, e);
      for (int t0 = lane * tb; t0 < e.qlen; t0 += 32 * tb) mine += tiles_of(e, t0);
    }
    if (mine) atomicAdd(&work, mine);
  }
  __syncthreads();
  int shift = 0;
  while ((top >> shift) >= kBuckets) ++shift;
  const int heads = p.Hkv * p.groups;
  const int share = (int)min((unsigned long long)(1 << 30),
                             (work * heads + 2 * fill - 1) / (unsigned long long)(2 * fill));
  const int longest = max(kMinPiece, share);
  auto pieces_of = [&](int tiles) { return cut ? max(1, (tiles + longest - 1) / longest) : 1; };
  auto bucket = [&](int tiles) { return kBuckets - 1 - (tiles >> shift); };  // 0: the longest
  for (int b = warp; b < p.B; b += 32) {
    Entry e;
    request(p, b, e);
    for (int t0 = lane * tb; t0 < e.qlen; t0 += 32 * tb) {
      const int tiles = tiles_of(e, t0), k = pieces_of(tiles);
      atomicAdd(&hist[bucket((tiles + k - 1) / k)], k);
    }
  }
  __syncthreads();
  {  // exclusive prefix of the buckets, two to a thread
    const int a = hist[2 * threadIdx.x], z = hist[2 * threadIdx.x + 1];
    int incl = a + z;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - a - z;
    for (int i = 0; i < warp; ++i) before += warp_sum[i];
    hist[2 * threadIdx.x] = before;
    hist[2 * threadIdx.x + 1] = before + a;
    if (threadIdx.x == 1023) count[0] = before + a + z;
  }
  __syncthreads();
  for (int b = warp; b < p.B; b += 32) {
    Entry e;
    request(p, b, e);
    e.pad[0] = e.pad[1] = e.pad[2] = 0;
    for (int t0 = lane * tb; t0 < e.qlen; t0 += 32 * tb) {
      const int tiles = tiles_of(e, t0), k = pieces_of(tiles), len = (tiles + k - 1) / k;
      const int at = atomicAdd(&hist[bucket(len)], k);
      e.t0 = t0;
      e.slot = -1;
      if (k > 1) {
        e.slot = atomicAdd(&n_slots, k);
        joins[atomicAdd(&n_joins, 1)] = Join{t0, e.q0, e.qlen, e.slot, k, {0, 0, 0}};
      }
      for (int i = 0; i < k; ++i) {
        Entry x = e;
        x.j0 = i * len;
        x.j1 = min(tiles, x.j0 + len);
        x.slot = k > 1 ? e.slot + i : -1;
        const int4* s = reinterpret_cast<const int4*>(&x);
        int4* d = reinterpret_cast<int4*>(list + at + i);
        d[0] = s[0];
        d[1] = s[1];
        d[2] = s[2];
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) count[1] = n_joins;
}

// Joins the pieces of an item,
//   lse = ln sum_i exp(lse_i),  out = sum_i exp(lse_i - lse) out_i:
// a thread per row and 16 columns, the rows of a warp side by side.  (8 columns
// and a quarter of the blocks: chunk of four prompts 187 us, replayed, now 179.)
constexpr int kJoinThreads = 128, kJoinColumns = 16;

template <int DV>
__global__ void __launch_bounds__(kJoinThreads) kv_prefill_join_kernel(const Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int heads = p.Hkv * p.groups, n = p.count[1];
  constexpr int kN = kJoinColumns, kC = DV / kN;  // kC threads to a row
  const int rows = p.rows_slot;
  for (int x = blockIdx.x; x < n * heads; x += gridDim.x) {
    const Join jn = p.joins[x / heads];
    const int h = x % heads, hk = h / p.groups, rg = h - hk * p.groups;
    for (int e = blockIdx.y * kJoinThreads + threadIdx.x; e < rows * kC;
         e += gridDim.y * kJoinThreads) {
      const int c = e / rows, row = e - c * rows;  // the rows of a warp lie side by side
      const int tok = jn.t0 + row / p.gg, head = rg * p.gg + row % p.gg;
      if (tok >= jn.qlen || head >= p.g) continue;
      const float* l = p.part_l + ((int64_t)jn.slot * heads + h) * rows + row;
      const float4* o = reinterpret_cast<const float4*>(p.part_o) +
                        (((int64_t)jn.slot * heads + h) * (DV / 4) + kN / 4 * c) * rows + row;
      const int64_t step = (int64_t)heads * rows;  // between two pieces
      float top = -INFINITY;
      for (int i = 0; i < jn.pieces; ++i) top = fmaxf(top, l[i * step]);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f, acc[kN];
#pragma unroll
      for (int k = 0; k < kN; ++k) acc[k] = 0.f;
#pragma unroll 2
      for (int i = 0; i < jn.pieces; ++i) {
        const float w = expf(l[i * step] - ref);
        sum += w;
#pragma unroll
        for (int k = 0; k < kN; k += 4) {
          const float4 a = o[i * step * (DV / 4) + k / 4 * rows];
          acc[k] = fmaf(w, a.x, acc[k]);
          acc[k + 1] = fmaf(w, a.y, acc[k + 1]);
          acc[k + 2] = fmaf(w, a.z, acc[k + 2]);
          acc[k + 3] = fmaf(w, a.w, acc[k + 3]);
        }
      }
      const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : NAN);
#pragma unroll
      for (int k = 0; k < kN; ++k) acc[k] *= inv;
      const int64_t off = (int64_t)(jn.q0 + tok) * p.o_st + (int64_t)(hk * p.g + head) * p.o_sh +
                          kN * c;
      if (p.out_dtype == TPLA_F32) {
        float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + off);
#pragma unroll
        for (int k = 0; k < kN; k += 4)
          d[k / 4] = make_float4(acc[k], acc[k + 1], acc[k + 2], acc[k + 3]);
      } else {
        uint32_t v[kN / 2];
#pragma unroll
        for (int k = 0; k < kN / 2; ++k)
          v[k] = p.out_dtype == TPLA_F16 ? F16::pack(acc[2 * k], acc[2 * k + 1])
                                         : Bf16::pack(acc[2 * k], acc[2 * k + 1]);
        uint16_t* const d = reinterpret_cast<uint16_t*>(p.out) + off;
        if (p.out32) {
          st_global_v8(d, v);
        } else {
          *reinterpret_cast<uint4*>(d) = make_uint4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<uint4*>(d + 8) = make_uint4(v[4], v[5], v[6], v[7]);
        }
      }
      if (p.lse && c == 0)
        p.lse[(int64_t)(jn.q0 + tok) * p.l_st + (int64_t)(hk * p.g + head) * p.l_sh] =
            sum > 0.f ? ref + logf(sum) : (sum == 0.f ? -INFINITY : NAN);
    }
  }
}

// ---------------------------------------------------------------- host side

struct Shape {
  int g, gg, groups, tpt, heads, sms;
  int64_t entries;  // most items of a head: ceil(T_b / (2 tpt)) summed over the requests
  bool planned;     // the list of items is made by the plan kernel
  int slots;        // partial results (times the heads) of items in pieces, 0: none are cut
  int rows_slot;
  int64_t capacity; // entries of the list
  int paired;
  size_t list_bytes, join_bytes, o_bytes, l_bytes;
};

Shape shape(const KvPrefillProblem& p, int sms) {
  Shape s;
  s.g = p.Hq / p.kv.Hkv;
  s.gg = s.g < kRows ? s.g : kRows;
  s.groups = (s.g + s.gg - 1) / s.gg;
  s.tpt = kRows / s.gg;
  s.heads = p.kv.Hkv * s.groups;
  s.sms = sms;
  s.entries = (int64_t)p.T / (2 * s.tpt) + p.B;
  // Items are cut where full ones would not go round the GPU twice and the
  // keys are long enough for two pieces.  No piece is longer than half a
  // block's share of the work, which bounds the pieces: see the plan kernel.
  const bool cut = (int64_t)p.T / (2 * s.tpt) * s.heads < 2 * sms &&
                   p.kv.cap_rows >= 2 * kMinPiece * kKeys;
  s.planned = p.B > 1 || cut;
  s.slots = cut ? (4 * sms + s.heads - 1) / s.heads : 0;
  s.rows_slot = (p.T < 2 * s.tpt ? p.T : 2 * s.tpt) * s.gg;
  s.capacity = s.entries + (cut ? 2 * sms : 0);
  // All heads' longest items first would have every head's keys and values in
  // use at once.  Where the L2 (126 MB) does not keep those, the items of one
  // prompt go head after head in pairs; the last round of pairs must be nearly
  // full, because a pair is up to twice an item.  128 heads of 4096 tokens
  // (335 MB of keys and values), replayed: 728 us longest first, 648 in pairs.
  // Calls of several prompts keep the longest-first order.
  const int64_t pairs = ((s.entries - p.B + 1) / 2) * s.heads, rounds = (pairs + sms - 1) / sms;
  s.paired = !s.planned && pairs > 0 && rounds * sms <= pairs + pairs / 16 &&
             p.kv.cap_rows * (p.kv.Dk + p.kv.Dv) * 2 * p.kv.Hkv > kL2Share;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  s.list_bytes = up((size_t)s.capacity * sizeof(Entry));
  s.join_bytes = up((size_t)s.slots * sizeof(Join));
  const size_t rows = (size_t)s.slots * s.heads * s.rows_slot;
  s.o_bytes = up(rows * p.kv.Dv * sizeof(float));
  s.l_bytes = up(rows * sizeof(float));
  return s;
}

template <typename T, int DK, int DV>
cudaError_t launch(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                   const Params& p, int slots, int grid, int dev, cudaStream_t stream) {
  using C = Cfg<T, DK, DV>;
  static std::mutex mu;
  static uint64_t ready = 0;  // devices whose shared-memory limit is raised
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(ready >> dev & 1)) {
      cudaError_t e = cudaFuncSetAttribute(kv_prefill_kernel<T, DK, DV>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (e != cudaSuccess) return e;
      ready |= 1ull << dev;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.count ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_prefill_kernel<T, DK, DV>, qm, km, vm, p);
  count_launch();
  if (e != cudaSuccess || !p.part_o) return e;
  // an item has two pieces or more; two runs of columns a thread
  const int runs = p.rows_slot * (DV / kJoinColumns);
  cfg.gridDim = dim3((unsigned)((slots * p.Hkv * p.groups + 1) / 2),
                     (unsigned)((runs + 2 * kJoinThreads - 1) / (2 * kJoinThreads)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, kv_prefill_join_kernel<DV>, p);
  count_launch();
  return e;
}

template <typename T>
cudaError_t launch_type(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                        const Params& p, int dk, int dv, int slots, int grid, int dev,
                        cudaStream_t stream) {
  if (dk == 64 && dv == 64) return launch<T, 64, 64>(qm, km, vm, p, slots, grid, dev, stream);
  if (dk == 128 && dv == 128) return launch<T, 128, 128>(qm, km, vm, p, slots, grid, dev, stream);
  if (dk == 192 && dv == 128) return launch<T, 192, 128>(qm, km, vm, p, slots, grid, dev, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

size_t kv_prefill_workspace_bytes(const KvPrefillProblem& p) {
  const Shape s = shape(p, sm_count(current_device()));
  return s.planned ? 256 + s.list_bytes + s.join_bytes + s.o_bytes + s.l_bytes : 0;
}

cudaError_t launch_kv_prefill(const KvPrefillProblem& dp, void* ws, cudaStream_t stream) {
  const int dev = current_device();
  if (!sm100_device(dev)) return cudaErrorNotSupported;
  const KvSource& kv = dp.kv;
  const Shape s = shape(dp, sm_count(dev));
  CUtensorMap qm, km, vm;
  {
    const cuuint64_t dims[5] = {64, (cuuint64_t)s.g, (cuuint64_t)dp.T, (cuuint64_t)(kv.Dk / 64),
                                (cuuint64_t)kv.Hkv};
    const cuuint64_t strides[4] = {map_stride(s.g, dp.q_sh), map_stride(dp.T, dp.q_st), 128,
                                   map_stride(kv.Hkv, dp.q_sh * s.g)};
    const cuuint32_t box[5] = {64, (cuuint32_t)s.gg, (cuuint32_t)s.tpt, 1, 1};
    if (!encode_16bit_5d(&qm, dp.q, kv.f16, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const int64_t rows = kv.page_table ? kBlock : kv.cap_rows;
  if (!encode_kv_tiles(&km, kv.k, dp.q, kv.f16, rows, kv.Hkv, kv.num_blocks, kv.k_s0, kv.k_s1,
                       kv.k_s2, kv.Dk, 1) ||
      !encode_kv_tiles(&vm, kv.v, dp.q, kv.f16, rows, kv.Hkv, kv.num_blocks, kv.v_s0, kv.v_s1,
                       kv.v_s2, kv.Dv, 1))
    return cudaErrorInvalidValue;
  Params p{};
  p.cu_q = dp.cu_q;
  p.cu_k = dp.cu_k;
  p.seq_lens = kv.seq_lens;
  p.page_table = kv.page_table;
  p.pt_sb = kv.pt_sb;
  p.num_blocks = (int)kv.num_blocks;
  p.cap_rows = (int)kv.cap_rows;
  p.B = dp.B;
  p.T = dp.T;
  p.Hkv = kv.Hkv;
  p.g = s.g;
  p.gg = s.gg;
  p.groups = s.groups;
  p.tpt = s.tpt;
  p.causal = dp.causal;
  // The row maximum is taken of the raw scores, negated for a negative scale.
  // A zero scale becomes f32's least number, 2^-149: masked scores (-inf) still
  // weigh 0, and the largest product there is, 2^128, moves a weight by 2^-21.
  const float scale_log2 = (float)(fabs((double)dp.scale) * 1.4426950408889634);
  p.scale_log2 = scale_log2 > 0.f ? scale_log2 : 0x1p-149f;
  p.negate = dp.scale < 0.f;
  p.out = dp.out;
  p.out_dtype = dp.out_dtype;
  p.o_st = dp.o_st;
  p.o_sh = dp.o_sh;
  p.lse = dp.lse;
  p.l_st = dp.l_st;
  p.l_sh = dp.l_sh;
  p.out32 = dp.out_dtype != TPLA_F32 && (reinterpret_cast<uintptr_t>(dp.out) & 31) == 0 &&
            (dp.T == 1 || dp.o_st % 16 == 0) && (dp.Hq == 1 || dp.o_sh % 16 == 0);
  p.rows_slot = s.rows_slot;
  p.paired = s.paired;
  const int64_t items = s.capacity * s.heads;
  if (items > (1LL << 31) - 1 - s.sms) return cudaErrorInvalidValue;
  if (s.planned) {
    char* at = reinterpret_cast<char*>(ws);
    int* count = reinterpret_cast<int*>(at);
    Entry* list = reinterpret_cast<Entry*>(at + 256);
    Join* joins = reinterpret_cast<Join*>(at + 256 + s.list_bytes);
    kv_prefill_plan_kernel<<<1, 1024, 0, stream>>>(p, list, joins, count, (int)s.entries,
                                                   s.slots > 0, s.sms);
    count_launch();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.count = count;
    p.list = list;
    p.joins = joins;
    if (s.slots > 0) {
      p.part_o = reinterpret_cast<float*>(at + 256 + s.list_bytes + s.join_bytes);
      p.part_l =
          reinterpret_cast<float*>(at + 256 + s.list_bytes + s.join_bytes + s.o_bytes);
    }
  }
  const int grid = (int)(items < s.sms ? items : s.sms);
  return kv.f16 ? launch_type<F16>(qm, km, vm, p, kv.Dk, kv.Dv, s.slots, grid, dev, stream)
                : launch_type<Bf16>(qm, km, vm, p, kv.Dk, kv.Dv, s.slots, grid, dev, stream);
}

cudaError_t status_read_clear_kv_prefill(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_prefill_status, sizeof(int));
  if (e != cudaSuccess) return e;
  if (v != 0) {
    int zero = 0;
    e = cudaMemcpyToSymbol(g_kv_prefill_status, &zero, sizeof(int));
  }
  *code = v;
  return e;
}

}  // namespace tpla
