// Decode attention of one new token per request over uncompressed keys and
// values, with grouped heads:
//   s_t = scale q[b,h] . k[b,t,h/g],  out = sum_t softmax(s)_t v[b,t,h/g],
//   lse = ln sum_t exp(s_t),          g = Hq / Hkv query heads to a key head.
//
// Bytes bound it: every cached value is read once for at most 2 g multiply-adds.
// The work is a row of units, request by request and key head by key head:
// the 64-token pages of a (request, head) and before them kSegUnits for its
// fixed work (queries, joining the warps).  Every SM takes an equal slice of
// that row, whatever the lengths, and a (request, head) that a slice's border
// cuts leaves normalised partial results that the merge kernel joins by their
// log-sum-exp.
//
// A block is eight consumer warps and TMA producer warps over rings of
// 64-token stages (K and V of one page of one key head, 128-byte swizzle).
// The g query heads are the rows of one or more 16-row matrix products
// (mma.sync m16n8k16: up to 16 rows a page gives the tensor core too little
// work to gain from TMEM accumulators, and the copies are the limit; with more
// rows every 16 of them read the page from shared memory again, see the figures
// for g > 16 below).  Warps split rows (16
// each, for g > 16) and then tokens; each keeps its own running maximum, sums
// and accumulator in registers, so nothing in the loop waits for another
// warp, and they meet once at the end of a (request, head) segment.  Up to 16
// rows the consumers are two groups of four warps, each with its slice, its
// ring and its producer: one group's segment end passes while the other reads.
//
// Measured (B200, the public Python call on data that the L2 does not hold;
// bytes of the cache against a copy's 6542 GB/s): 4 requests of 131072 tokens, 64
// heads over 8 of 128: 321 us, 6.7 TB/s, 102 %; 32 of 2048 to 4096, 32 over 8: 76
// us, 83 %; 13 ragged ones of 16 heads, 192 / 128, f16: 72 us, 76 % (the slices'
// ends: start, last page, joins, merge); 1 of 256 tokens: 10.3 us, nearly all
// fixed (in a replayed graph 8.6: start 2, one page 2.5, join 0.7, merge launch
// and read 1.5).  32 requests of 2048 to 4063 tokens, 8 key heads of 128, by g: 1:
// 73 us; 4: 74; 16: 77; 17: 97; 32: 99; 33: 152; 64: 157; 65: 361; 128: 368 (192 /
// 128: 95, 96, 100, 119, 122, 174, 183, 308, 320).  From 17 rows on the copies (61
// and 77 us) bound it no longer.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "internal.h"
#include "kv_map.h"
#include "kv_ptx.cuh"

namespace tpla {
namespace {

using namespace kvx;

__device__ int g_kv_decode_status;

constexpr int kPage = 64;
constexpr int kConsumers = 8;                      // warps
constexpr int kMaxRows = 128;                      // query heads of one row group
constexpr int kMaxStages = 12;
// 13 ragged requests of 16 heads in a replayed graph: 94, 87, 71, 68, 68 us for 0 to 4
constexpr int kSegUnits = 3;
constexpr int kSmemMax = 232448;
constexpr int kMiscBytes = 2560;                   // barriers, stage counts, statistics

struct Params {
  const uint16_t* q;
  int64_t q_sb, q_sh;
  const int* seq_lens;
  const int* page_table;
  int64_t pt_sb;
  int64_t num_blocks;
  int cap_rows;
  int B, Hq, Hkv, g, groups, rows;  // row groups per key head, rows of a group (<= 128)
  float scale_log2;
  int ranges;                       // slices of the work (one a group of warps)
  void* out;
  int out_dtype;
  int64_t o_sb, o_sh;
  float* lse;
  int64_t l_sb, l_sh;
  int4* cut;        // [ranges] the task that slice r begins and does not end:
                    // (first slot, pieces, request, task), pieces 0: none
  float* part_o;    // [2 ranges, rows, Dv]
  float* part_l;    // [2 ranges, rows]
};

__device__ __forceinline__ int req_len(const Params& p, int b) {
  const int n = p.seq_lens[b];
  if (n < 0 || n > p.cap_rows) {
    atomicCAS(&g_kv_decode_status, 0, TPLA_ERR_DEVICE_BOUNDS);
    return n < 0 ? 0 : p.cap_rows;
  }
  return n;
}

__device__ __forceinline__ int req_pages(const Params& p, int b) {
  return (req_len(p, b) + kPage - 1) / kPage;
}

__device__ __forceinline__ long long req_units(const Params& p, int b) {
  const int pages = req_pages(p, b);
  return pages ? (long long)(pages + kSegUnits) * p.Hkv * p.groups : 0;
}

// Where a slice stands in the row of units.
struct Walk {
  int b;
  long long base;  // units before request b
  long long pos, hi;
  int emitted;     // segments so far
};

struct Segment {
  int b, task, page0, page1, len;
  int complete, slot;
  long long end;   // unit behind the task
};

// The slice's next segment: a slice cuts at most its first and its last, so
// two slots a slice hold what is not complete.
__device__ __forceinline__ bool seg_next(const Params& p, int range, Walk& w, Segment& s) {
  const int tasks = p.Hkv * p.groups;
  while (w.pos < w.hi) {
    const int len = req_len(p, w.b);
    const int pages = (len + kPage - 1) / kPage, units = pages + kSegUnits;
    const long long n = pages ? (long long)units * tasks : 0;
    if (w.pos >= w.base + n) {
      w.base += n;
      ++w.b;
      continue;
    }
    const long long off = w.pos - w.base;
    s.b = w.b;
    s.len = len;
    s.task = off >> 32 ? (int)(off / units) : (int)((uint32_t)off / (uint32_t)units);
    const int u0 = (int)(off - (long long)s.task * units);
    const long long left = w.hi - w.pos;
    const int u1 = left < units - u0 ? u0 + (int)left : units;
    w.pos += u1 - u0;
    s.page0 = max(u0 - kSegUnits, 0);
    s.page1 = u1 - kSegUnits;
    if (s.page1 <= s.page0) continue;  // the slice ends in the fixed work
    s.complete = s.page0 == 0 && s.page1 == pages;
    s.slot = 2 * range + (w.emitted ? 1 : 0);
    s.end = w.base + (long long)(s.task + 1) * units;
    ++w.emitted;
    return true;
  }
  return false;
}

__device__ __forceinline__ void store_out(const Params& p, int b, int h, int c, float v0, float v1) {
  const int64_t off = (int64_t)b * p.o_sb + (int64_t)h * p.o_sh + c;
  if (p.out_dtype == TPLA_F32) {
    *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.out) + off) = make_float2(v0, v1);
  } else {
    *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + off) =
        p.out_dtype == TPLA_F16 ? F16::pack(v0, v1) : Bf16::pack(v0, v1);
  }
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<Bf16>(float (&c)[4], const uint32_t* a, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<F16>(float (&c)[4], const uint32_t* a, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Byte offset of 16-byte column c16 of row `row` in a tile of 64-row,
// 128-byte swizzled chunks of 64 columns.
__device__ __forceinline__ uint32_t tile_off(int row, int c16) {
  return (uint32_t)((c16 >> 3) * 8192 + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
}

// DK, DV: head widths; RB: 16-row blocks of the row group (1, 2, 4, 8).
template <typename T, int DK, int DV, int RB>
struct Cfg {
  static constexpr int kGroups = RB == 1 ? 2 : 1;        // of warps, each with a slice of its own
  static constexpr int kWarps = kConsumers / kGroups;    // consumers of a group
  static constexpr int kThreads = 32 * (kConsumers + kGroups);
  static constexpr int kK = kPage * DK * 2, kV = kPage * DV * 2;
  static constexpr int kStage = kK + kV;
  static constexpr int kTS = kWarps / RB;                // warps that share a row block: token slices
  static constexpr int kNT = kPage / kTS;                // tokens of a slice
  static constexpr int kJoin = kWarps * 16 * (DV / 2) * 4;  // one half of the columns
  static constexpr int kRing0 =
      (kSmemMax - kMiscBytes - kGroups * kJoin) / kStage / kGroups;
  static constexpr int kStages = kRing0 < kMaxStages ? kRing0 : kMaxStages;  // of a group
  static constexpr int kSmem = kGroups * (kStages * kStage + kJoin) + kMiscBytes;
  static_assert(kStages >= 2 && kSmem <= kSmemMax, "shared memory");
};

struct GroupMisc {  // in shared memory
  unsigned long long full[kMaxStages], empty[kMaxStages];
  int nv[kMaxStages];  // valid tokens of a stage
  int b0;
  long long base0;
};
struct Misc {
  GroupMisc group[2];
  int abort_flag;
  long long warp_sum[kConsumers + 2];
  float stat[kConsumers][16][3];  // m, sum of rounded weights, sum of exact weights
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc shared memory");

template <typename T, int DK, int DV, int RB>
__global__ void __launch_bounds__(Cfg<T, DK, DV, RB>::kThreads, 1)
kv_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const Params p) {
  using C = Cfg<T, DK, DV, RB>;
  extern __shared__ __align__(1024) uint8_t smem[];  // swizzled tiles begin on 1 KB
  Misc& all = *reinterpret_cast<Misc*>(smem + C::kGroups * (C::kStages * C::kStage + C::kJoin));
  volatile int* abort_flag = &all.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // consumers of group 0, of group 1, then the producers
  const bool produces = warp >= kConsumers;
  const int group = produces ? warp - kConsumers : warp / C::kWarps;
  const int range = blockIdx.x * C::kGroups + group;
  GroupMisc& ms = all.group[group];
  const uint32_t sbase = smem_addr(smem + group * C::kStages * C::kStage);
  float* join = reinterpret_cast<float*>(smem + C::kGroups * C::kStages * C::kStage +
                                         group * C::kJoin);

  if (threadIdx.x == 0) {
    for (int g = 0; g < C::kGroups; ++g)
      for (int i = 0; i < C::kStages; ++i) {
        mbar_init(smem_addr(&all.group[g].full[i]), 1);
        mbar_init(smem_addr(&all.group[g].empty[i]), C::kWarps);
      }
    all.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kConsumers && lane == 0) {
    tma_prefetch(&kmap);
    tma_prefetch(&vmap);
  }
  // the merge may be launched beside this kernel: it waits for its end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // units before each thread's run of requests, and the request where this
  // block's slice begins
  const int run = (p.B + C::kThreads - 1) / C::kThreads;
  const int b_lo = min(p.B, (int)threadIdx.x * run), b_hi = min(p.B, b_lo + run);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += req_units(p, b);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) all.warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kConsumers + C::kGroups; ++i) {
    if (i < warp) before += all.warp_sum[i];
    total += all.warp_sum[i];
  }
  // no slice is empty: where there are fewer units than groups, the first
  // `slices` groups take one each
  const long long slices = total < p.ranges ? total : p.ranges;
  auto slice_begin = [&](int r) { return r < slices ? total * r / slices : total; };
#pragma unroll
  for (int g = 0; g < C::kGroups; ++g) {
    const long long at = slice_begin(blockIdx.x * C::kGroups + g);
    if (at >= before && at < before + mine) {
      long long base = before;
      int b = b_lo;
      for (;; ++b) {
        const long long n = req_units(p, b);
        if (at < base + n) break;
        base += n;
      }
      all.group[g].b0 = b;
      all.group[g].base0 = base;
    }
  }
  Walk w;
  w.pos = slice_begin(range);
  w.hi = slice_begin(range + 1);
  w.emitted = 0;
  // requests without tokens
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (req_pages(p, b) > 0) continue;
    for (int e = threadIdx.x; e < p.Hq * (DV / 2); e += C::kThreads) {
      const int h = e / (DV / 2), c = 2 * (e - h * (DV / 2));
      store_out(p, b, h, c, 0.f, 0.f);
      if (c == 0 && p.lse) p.lse[(int64_t)b * p.l_sb + (int64_t)h * p.l_sh] = -INFINITY;
    }
  }
  __syncthreads();
  if (w.pos >= w.hi) {
    if (!produces && warp == group * C::kWarps && lane == 0 && range < p.ranges)
      p.cut[range] = make_int4(0, 0, 0, 0);
    return;
  }
  w.b = ms.b0;
  w.base = ms.base0;
  Segment s;
  uint32_t n = 0;  // stages so far

  if (produces) {  // ------------------------------------------------------- producer
    int ok = 1;
    while (ok && seg_next(p, range, w, s)) {
      const int hk = s.task / p.groups;
      int win = 0;  // lane i: page id of page w0 + i
      for (int pg = s.page0, w0 = pg; pg < s.page1; ++pg, ++n) {
        if (p.page_table && ((pg - w0) & 31) == 0) {
          w0 = pg;
          win = pg + lane < s.page1 ? p.page_table[(int64_t)s.b * p.pt_sb + pg + lane] : 0;
        }
        const int blk = p.page_table ? __shfl_sync(0xffffffffu, win, pg - w0) : s.b;
        const int slot = n % C::kStages;
        if (lane == 0 && n >= C::kStages)
          ok = wait_bar(smem_addr(&ms.empty[slot]), ((n / C::kStages) - 1) & 1, abort_flag,
                        &g_kv_decode_status);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane == 0) {
          const int row = p.page_table ? 0 : pg * kPage;
          const uint32_t full = smem_addr(&ms.full[slot]);
          const uint32_t dst = sbase + slot * C::kStage;
          if (blk < 0 || blk >= p.num_blocks) {
            atomicCAS(&g_kv_decode_status, 0, TPLA_ERR_DEVICE_BOUNDS);
            ms.nv[slot] = 0;
            arrive(full);
          } else {
            ms.nv[slot] = min(kPage, s.len - pg * kPage);
            mbar_arrive_expect_tx(full, C::kStage);
            tma_load_5d(dst, &kmap, 0, row, 0, hk, blk, full);
            tma_load_5d(dst + C::kK, &vmap, 0, row, 0, hk, blk, full);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) {  // no copy outlives the block, whatever its consumers do
      const long long since = clock64();
      for (uint32_t i = n < C::kStages ? 0 : n - C::kStages; i < n; ++i)
        wait_landed(smem_addr(&ms.full[i % C::kStages]), (i / C::kStages) & 1, since);
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int gw = warp - group * C::kWarps, tid = gw * 32 + lane;  // within the group
  const int rb = gw % RB, slice = gw / RB;
  const int r = lane >> 2, c2 = (lane & 3) * 2;
  const int t0 = slice * C::kNT;
  const uint32_t bar_id = 1 + group;
  float(*stat)[16][3] = all.stat + group * C::kWarps;  // of the group's warps
  bool dead = false;  // a wait gave up: no more pages, but the block's barriers are kept
  // the queries as A fragments: rows r and r + 8 of this row block
  uint32_t qf[DK / 16][4];
  const int row = rb * 16 + r;
  auto load_q = [&](const Segment& sg) {
    const int hk = sg.task / p.groups, rg = sg.task - hk * p.groups;
    const int nrows = min(p.g - rg * kMaxRows, kMaxRows);
    const uint16_t* q0 = p.q + (int64_t)sg.b * p.q_sb +
                         (int64_t)(hk * p.g + rg * kMaxRows + row) * p.q_sh + c2;
    const uint16_t* q1 = q0 + 8 * p.q_sh;
#pragma unroll
    for (int k = 0; k < DK / 16; ++k) {
      qf[k][0] = row < nrows ? *reinterpret_cast<const uint32_t*>(q0 + 16 * k) : 0u;
      qf[k][1] = row + 8 < nrows ? *reinterpret_cast<const uint32_t*>(q1 + 16 * k) : 0u;
      qf[k][2] = row < nrows ? *reinterpret_cast<const uint32_t*>(q0 + 16 * k + 8) : 0u;
      qf[k][3] = row + 8 < nrows ? *reinterpret_cast<const uint32_t*>(q1 + 16 * k + 8) : 0u;
    }
  };
  Segment nx;
  bool more = seg_next(p, range, w, nx);
  if (more) load_q(nx);
  if (tid == 0) p.cut[range] = make_int4(0, 0, 0, 0);
  while (more) {
    s = nx;
    more = seg_next(p, range, w, nx);
    const int hk = s.task / p.groups, rg = s.task - hk * p.groups;
    const int h0 = hk * p.g + rg * kMaxRows;            // first head of the row group
    const int nrows = min(p.g - rg * kMaxRows, kMaxRows);
    if (tid == 0 && !s.complete && s.page0 == 0) {
      // the slice with the task's last page
      const int last = total < (1 << 22)  // times at most 2^9 slices
                           ? (int)(((uint32_t)s.end * (uint32_t)slices - 1) / (uint32_t)total)
                           : (int)((s.end * slices - 1) / total);
      p.cut[range] = make_int4(s.slot, last - range + 1, s.b, s.task);
    }
    float o[DV / 8][4];
#pragma unroll
    for (int i = 0; i < DV / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY};  // running maximum of the scaled scores, log2 units
    // both lifted by T::kLift
    float lr[2] = {0.f, 0.f};             // sum of the 16-bit weights: normalises the output
    float le[2] = {0.f, 0.f};             // sum of the f32 weights: the log-sum-exp

    for (int pg = dead ? s.page1 : s.page0; pg < s.page1; ++pg, ++n) {
      const int slot = n % C::kStages;
      int ok = 1;
      if (lane == 0)
        ok = wait_bar(smem_addr(&ms.full[slot]), (n / C::kStages) & 1, abort_flag,
                      &g_kv_decode_status);
      if (!__shfl_sync(0xffffffffu, ok, 0)) {
        dead = true;
        break;
      }
      __syncwarp();
      const int nv = ms.nv[slot] - t0;  // valid tokens of the slice
      if (nv > 0) {
        const uint32_t kt = sbase + slot * C::kStage, vt = kt + C::kK;
        float sc[C::kNT / 8][4];
#pragma unroll
        for (int i = 0; i < C::kNT / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll
        for (int k = 0; k < DK / 32; ++k) {
#pragma unroll
          for (int i = 0; i < C::kNT / 8; ++i) {
            uint32_t f[4];
            ldsm4(kt + tile_off(t0 + 8 * i + (lane & 7), 4 * k + (lane >> 3)), f);
            mma16816<T>(sc[i], qf[2 * k], f[0], f[1]);
            mma16816<T>(sc[i], qf[2 * k + 1], f[2], f[3]);
          }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < C::kNT / 8; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = sc[i][j] * p.scale_log2;
            sc[i][j] = 8 * i + c2 + (j & 1) < nv ? x : -INFINITY;
            mx[j >> 1] = fmaxf(mx[j >> 1], sc[i][j]);
          }
        }
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 1));
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 2));
          const float mn = fmaxf(m[j], mx[j]);
          f[j] = m[j] == mn ? 1.f : ex2(m[j] - mn);
          m[j] = mn;
          lr[j] *= f[j];
          le[j] *= f[j];
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < DV / 8; ++i) {
            o[i][0] *= f[0];
            o[i][1] *= f[0];
            o[i][2] *= f[1];
            o[i][3] *= f[1];
          }
        }
        const float ms0 = m[0] == -INFINITY ? 0.f : m[0] - T::kLift;
        const float ms1 = m[1] == -INFINITY ? 0.f : m[1] - T::kLift;
#pragma unroll
        for (int k = 0; k < C::kNT / 16; ++k) {
          uint32_t a[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // a[0], a[2]: row r; a[1], a[3]: row r + 8
            float* x = sc[2 * k + (j >> 1)] + 2 * (j & 1);
            const float e0 = ex2(x[0] - (j & 1 ? ms1 : ms0)), e1 = ex2(x[1] - (j & 1 ? ms1 : ms0));
            le[j & 1] += e0 + e1;
            a[j] = T::pack(e0, e1);
            const float2 e = T::unpack(a[j]);
            lr[j & 1] += e.x + e.y;
          }
          const bool whole = nv >= 16 * (k + 1);
          // tokens of this lane's B fragments: 16 k + c2 + {0, 1} and + 8
          const uint32_t keep0 = (16 * k + c2 < nv ? 0xffffu : 0u) |
                                 (16 * k + c2 + 1 < nv ? 0xffff0000u : 0u);
          const uint32_t keep1 = (16 * k + c2 + 8 < nv ? 0xffffu : 0u) |
                                 (16 * k + c2 + 9 < nv ? 0xffff0000u : 0u);
#pragma unroll
          for (int i = 0; i < DV / 16; ++i) {
            uint32_t v[4];
            ldsm4t(vt + tile_off(t0 + 16 * k + (lane & 15), 2 * i + (lane >> 4)), v);
            if (!whole) {  // what stands behind the last token is not multiplied
              v[0] &= keep0;
              v[1] &= keep1;
              v[2] &= keep0;
              v[3] &= keep1;
            }
            mma16816<T>(o[2 * i], a, v[0], v[1]);
            mma16816<T>(o[2 * i + 1], a, v[2], v[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) arrive(smem_addr(&ms.empty[slot]));
    }

    if (more) load_q(nx);  // on their way while the warps join
    // join the warps that share a row block
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        lr[j] += __shfl_xor_sync(0xffffffffu, lr[j], x);
        le[j] += __shfl_xor_sync(0xffffffffu, le[j], x);
      }
      if ((lane & 3) == 0) {
        float* st = stat[gw][r + 8 * j];
        st[0] = m[j];
        st[1] = lr[j];
        st[2] = le[j];
      }
    }
    named_bar_sync(bar_id, 32 * C::kWarps);
    // this warp's factor in its rows' results, and the rows' log-sum-exp
    float f[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int ri = r + 8 * j;
      float top = -INFINITY, slr = 0.f, sle = 0.f;
#pragma unroll
      for (int x = 0; x < C::kTS; ++x) top = fmaxf(top, stat[x * RB + rb][ri][0]);
#pragma unroll
      for (int x = 0; x < C::kTS; ++x) {
        const float* st = stat[x * RB + rb][ri];
        const float fx = st[0] == -INFINITY ? 0.f : ex2(st[0] - top);
        slr += st[1] * fx;
        sle += st[2] * fx;
      }
      const float inv = slr > 0.f ? 1.f / slr : (slr == 0.f ? 0.f : NAN);
      f[j] = m[j] == -INFINITY ? 0.f : ex2(m[j] - top) * inv;
      const int rw = rb * 16 + ri;
      if (slice == 0 && (lane & 3) == 0 && rw < nrows) {
        const float l = sle > 0.f ? (top + (log2f(sle) - T::kLift)) * kLn2 : (sle == 0.f ? -INFINITY : NAN);
        if (!s.complete)
          p.part_l[(int64_t)s.slot * p.rows + rw] = l;
        else if (p.lse)
          p.lse[(int64_t)s.b * p.l_sb + (int64_t)(h0 + rw) * p.l_sh] = l;
      }
    }
    // all columns at once where the rows above 8 are not used, else in halves;
    // 8-column blocks change places by row, so that the rows' stores meet in
    // no bank
    const bool narrow = RB == 1 && nrows <= 8;
    const int passes = narrow ? 1 : 2, rows_w = narrow ? 8 : 16;
    const int cols = DV / passes;
    for (int pass = 0; pass < passes; ++pass) {
      if (pass) named_bar_sync(bar_id, 32 * C::kWarps);
      float* d = join + (gw * rows_w + r) * cols;
#pragma unroll
      for (int i = 0; i < DV / 8; ++i) {
        const int at = 8 * i - pass * cols;
        if (at < 0 || at >= cols) continue;
        const int c = (at ^ ((r & 3) << 3)) + c2;
        *reinterpret_cast<float2*>(d + c) = make_float2(o[i][0] * f[0], o[i][1] * f[0]);
        if (!narrow)
          *reinterpret_cast<float2*>(d + 8 * cols + c) =
              make_float2(o[i][2] * f[1], o[i][3] * f[1]);
      }
      named_bar_sync(bar_id, 32 * C::kWarps);
      for (int e = tid; e < nrows * (cols / 4); e += 32 * C::kWarps) {
        const int rw = e / (cols / 4), c = 4 * (e - rw * (cols / 4));
        const int blk = rw >> 4, ri = rw & 15;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < C::kTS; ++x) {
          const float4 y = *reinterpret_cast<const float4*>(
              join + ((x * RB + blk) * rows_w + ri) * cols + (c ^ ((ri & 3) << 3)));
          v.x += y.x;
          v.y += y.y;
          v.z += y.z;
          v.w += y.w;
        }
        const int col = pass * cols + c;
        if (s.complete) {
          store_out(p, s.b, h0 + rw, col, v.x, v.y);
          store_out(p, s.b, h0 + rw, col + 2, v.z, v.w);
        } else {
          *reinterpret_cast<float4*>(p.part_o + ((int64_t)s.slot * p.rows + rw) * DV + col) = v;
        }
      }
    }
    named_bar_sync(bar_id, 32 * C::kWarps);
  }
}

// ---------------------------------------------------------------- merge
// Joins the pieces of the tasks that a slice's border cuts: a warp per row, a
// block column per slice, which says what it began and did not end.  The
// following pieces are the first segments of the following slices.  (The code
// is short on purpose: fetching instructions is most of a small launch.)
constexpr int kMergeWarps = 4;

template <int DV>
__global__ void __launch_bounds__(32 * kMergeWarps) kv_decode_merge_kernel(const Params p) {
  const int rw = blockIdx.y * kMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int range = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 cut = p.cut[range];
  const int n = cut.y, hk = cut.w / p.groups, rg = cut.w - hk * p.groups;
  if (n == 0 || rw >= min(p.g - rg * kMaxRows, kMaxRows)) return;
  auto row_of = [&](int i) { return (i ? 2 * (range + i) : cut.x) * p.rows + rw; };
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, p.part_l[row_of(i)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -INFINITY ? 0.f : top;
  constexpr int kV = DV / 32;  // values of a lane
  float sum = 0.f, acc[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float wgt = ex2((p.part_l[row_of(i)] - ref) * kLog2e);
    const float* src = p.part_o + (int64_t)row_of(i) * DV + lane * kV;
    sum += wgt;
#pragma unroll
    for (int k = 0; k < kV; k += 2) {
      const float2 v = *reinterpret_cast<const float2*>(src + k);
      acc[k] = fmaf(wgt, v.x, acc[k]);
      acc[k + 1] = fmaf(wgt, v.y, acc[k + 1]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : NAN);
  const int h = hk * p.g + rg * kMaxRows + rw;
#pragma unroll
  for (int i = 0; i < kV; i += 2)
    store_out(p, cut.z, h, lane * kV + i, acc[i] * inv, acc[i + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[(int64_t)cut.z * p.l_sb + (int64_t)h * p.l_sh] =
        sum > 0.f ? ref + log2f(sum) * kLn2 : (sum == 0.f ? -INFINITY : NAN);
}

// ---------------------------------------------------------------- host side

template <typename T, int DK, int DV, int RB>
cudaError_t launch_rb(const CUtensorMap& km, const CUtensorMap& vm, const Params& p, int dev,
                      cudaStream_t stream) {
  using C = Cfg<T, DK, DV, RB>;
  static std::mutex mu;
  static uint64_t ready = 0;  // devices whose shared-memory limit is raised
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(ready >> dev & 1)) {
      cudaError_t e = cudaFuncSetAttribute(kv_decode_kernel<T, DK, DV, RB>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (e != cudaSuccess) return e;
      ready |= 1ull << dev;
    }
  }
  kv_decode_kernel<T, DK, DV, RB>
      <<<(p.ranges + C::kGroups - 1) / C::kGroups, C::kThreads, C::kSmem, stream>>>(km, vm, p);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ranges,
                     (unsigned)((p.rows + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_decode_merge_kernel<DV>, p);
  count_launch();
  return e;
}

template <typename T, int DK, int DV>
cudaError_t launch_dims(const CUtensorMap& km, const CUtensorMap& vm, const Params& p, int dev,
                        cudaStream_t stream) {
  if (p.rows <= 16) return launch_rb<T, DK, DV, 1>(km, vm, p, dev, stream);
  if (p.rows <= 32) return launch_rb<T, DK, DV, 2>(km, vm, p, dev, stream);
  if (p.rows <= 64) return launch_rb<T, DK, DV, 4>(km, vm, p, dev, stream);
  return launch_rb<T, DK, DV, 8>(km, vm, p, dev, stream);
}

template <typename T>
cudaError_t launch_type(const CUtensorMap& km, const CUtensorMap& vm, const Params& p, int dk,
                        int dv, int dev, cudaStream_t stream) {
  if (dk == 64 && dv == 64) return launch_dims<T, 64, 64>(km, vm, p, dev, stream);
  if (dk == 128 && dv == 128) return launch_dims<T, 128, 128>(km, vm, p, dev, stream);
  if (dk == 192 && dv == 128) return launch_dims<T, 192, 128>(km, vm, p, dev, stream);
  return cudaErrorInvalidValue;
}

struct Schedule {
  int g, groups, rows, ranges;
  size_t cut_bytes, o_bytes, l_bytes;
};

// One block per SM (it takes the SM's shared memory), and in it a slice for
// each group of warps; fewer where the caches cannot hold that many pages.
Schedule schedule(const KvDecodeProblem& p, int device) {
  Schedule s;
  s.g = p.Hq / p.kv.Hkv;
  s.groups = (s.g + kMaxRows - 1) / kMaxRows;
  s.rows = s.g < kMaxRows ? s.g : kMaxRows;
  const int sms = sm_count(device);
  const int64_t pages = (p.kv.cap_rows + kPage - 1) / kPage;
  const int64_t units = (pages + kSegUnits) * p.B * p.kv.Hkv * s.groups;
  const int most = s.rows <= 16 ? 2 * sms : sms;
  s.ranges = (int)(units < most ? (units > 0 ? units : 1) : most);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  s.cut_bytes = up((size_t)s.ranges * sizeof(int4));
  s.o_bytes = up((size_t)2 * s.ranges * s.rows * p.kv.Dv * sizeof(float));
  s.l_bytes = up((size_t)2 * s.ranges * s.rows * sizeof(float));
  return s;
}

}  // namespace

bool kv_head_dims_supported(int Dk, int Dv) {
  return (Dk == 64 && Dv == 64) || (Dk == 128 && Dv == 128) || (Dk == 192 && Dv == 128);
}

size_t kv_decode_workspace_bytes(const KvDecodeProblem& p, int device) {
  const Schedule s = schedule(p, device);
  return s.cut_bytes + s.o_bytes + s.l_bytes;
}

cudaError_t launch_kv_decode(const KvDecodeProblem& dp, void* ws, cudaStream_t stream) {
  const int dev = current_device();
  if (!sm100_device(dev)) return cudaErrorNotSupported;
  const Schedule s = schedule(dp, dev);
  const KvSource& kv = dp.kv;
  const int64_t rows = kv.page_table ? kPage : kv.cap_rows;
  CUtensorMap km, vm;
  if (!encode_kv_tiles(&km, kv.k, dp.q, kv.f16, rows, kv.Hkv, kv.num_blocks, kv.k_s0, kv.k_s1,
                       kv.k_s2, kv.Dk, kv.Dk / 64) ||
      !encode_kv_tiles(&vm, kv.v, dp.q, kv.f16, rows, kv.Hkv, kv.num_blocks, kv.v_s0, kv.v_s1,
                       kv.v_s2, kv.Dv, kv.Dv / 64))
    return cudaErrorInvalidValue;
  Params p{};
  p.q = reinterpret_cast<const uint16_t*>(dp.q);
  p.q_sb = dp.q_sb;
  p.q_sh = dp.q_sh;
  p.seq_lens = kv.seq_lens;
  p.page_table = kv.page_table;
  p.pt_sb = kv.pt_sb;
  p.num_blocks = kv.num_blocks;
  p.cap_rows = (int)kv.cap_rows;
  p.B = dp.B;
  p.Hq = dp.Hq;
  p.Hkv = kv.Hkv;
  p.g = s.g;
  p.groups = s.groups;
  p.rows = s.rows;
  p.scale_log2 = (float)((double)dp.scale * 1.4426950408889634);
  p.ranges = s.ranges;
  p.out = dp.out;
  p.out_dtype = dp.out_dtype;
  p.o_sb = dp.o_sb;
  p.o_sh = dp.o_sh;
  p.lse = dp.lse;
  p.l_sb = dp.l_sb;
  p.l_sh = dp.l_sh;
  char* at = reinterpret_cast<char*>(ws);
  p.cut = reinterpret_cast<int4*>(at);
  p.part_o = reinterpret_cast<float*>(at + s.cut_bytes);
  p.part_l = reinterpret_cast<float*>(at + s.cut_bytes + s.o_bytes);
  return kv.f16 ? launch_type<F16>(km, vm, p, kv.Dk, kv.Dv, dev, stream)
                : launch_type<Bf16>(km, vm, p, kv.Dk, kv.Dv, dev, stream);
}

cudaError_t status_read_clear_kv_decode(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_decode_status, sizeof(int));
  if (e != cudaSuccess) return e;
  if (v != 0) {
    int zero = 0;
    e = cudaMemcpyToSymbol(g_kv_decode_status, &zero, sizeof(int));
  }
  *code = v;
  return e;
}

}  // namespace tpla
