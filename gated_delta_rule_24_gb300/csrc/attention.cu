// Softmax attention of new tokens over a paged cache and a prefix that all sequences share, for sm_103a.
//
//   s_j = scale q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = log sum_j exp(s_j)
//
// The queries of one key head (tokens x group rows, 16 at a time) against a sequence's keys are a unit.
// A row's sums are kept relative to 2^base (base near the largest score so far, in powers of two):
// (base, sum of weights, sum of weighted values) of two sets of keys join into those of their union, so a
// unit can be cut anywhere.  All units' tiles of 64 keys, one unit behind the other, are cut into equal
// shares for as many workers (CTAs) as run at once, whatever the lengths are: a worker takes the end of one unit,
// some whole ones, and the beginning of another.  Whole units go to the output, the cut ones' parts to the workspace, and
// a second kernel joins those.
//
// Each key and value is read once for up to 16 rows, 2 x 16 flops a byte at most: the kernel is bound by
// HBM bandwidth as long as copies are always under way.  A warp of its own looks up pages and issues the tensor
// copies (boxes of up to 64 places of a page) into a ring of three tiles, over the ends of units; with a unit's first
// tile come its queries.  Four warps take 16 of a tile's keys each: scores and sums by warp products
// with the keys as the narrow side, weights passed on in registers.  They meet at the end of a unit only, over the
// memory of its last tile.
#include <cuda_runtime.h>

#include <algorithm>

#include "attention.h"
#include "decay.cuh"
#include "ptx.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;                      // that compute; one more copies
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kWarpKeys = 16, kTile = kWarps * kWarpKeys;
static_assert(kTile == kOwnKeys, "boxes fit a tile");
constexpr int kRows = 16;                      // rows of a unit
constexpr int kStages = 3;
constexpr int kHalfBytes = kTile * 128;        // 64 of a row's 128 values
constexpr int kTileBytes = 4 * kHalfBytes;     // keys, then values
constexpr int kQueryBytes = kRows * 256;
static_assert(kWarps * kRows * kHeadDim * 4 == kTileBytes, "the warps' sums lie over a tile");
struct Bars {
  float2 ml[kWarps][kRows];
  uint64_t full[kStages], empty[kStages];
  int64_t found[kWarps + 1];                   // the walk's start
  uint32_t bad[kStages];                       // a page of the stage's tile is none
};
constexpr int kSmemBytes = kStages * (kTileBytes + kQueryBytes) + sizeof(Bars);
constexpr int kResident = 2;                   // workers on an SM
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint64_t kWaitNs = 200000000ull;
constexpr float kRoom = 8.f;                   // how far (powers of two) scores may exceed the base before it moves
constexpr float kBad = kAttentionBad;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Kernels of a call are launched one behind the other without a gap: each lets the next start when it has started
// itself (go_ahead), and waits for the end of the one before it (grid_wait) before it reads what that has written, and before it
// ends.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void go_ahead() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Keys of sequence n in its own pages, or -1 where its length is none.
__device__ __forceinline__ int length_of(const AttentionParams& p, int n) {
  const int64_t x = index_at(p.lengths, p.len_dtype, n);
  return x < 0 || x > (int64_t)p.max_pages * p.page_size ? -1 : (int)x;
}
__device__ __forceinline__ int tiles_of(int length) { return length > 0 ? (length + kTile - 1) / kTile : 0; }

// A tile of the walk through all units: sequence n (N: the prefix), `sub` = key head * row blocks + row
// block, tile t.  The lanes of a warp hold the lengths of 32 sequences.
struct Walk {
  int n, sub, t, tiles, length, subs;
  int held, held_from;

  __device__ __forceinline__ void hold(const AttentionParams& p, int lane) {
    held_from = n;
    held = n + lane < p.N ? length_of(p, n + lane) : 0;
  }
  __device__ __forceinline__ void enter(const AttentionParams& p, int lane) {  // lengths of n, which has keys
    if (n >= p.N) {
      length = p.prefix;
      subs = p.H_k * p.prefix_blocks;
    } else {
      if (n - held_from >= 32) hold(p, lane);
      length = __shfl_sync(0xffffffffu, held, n - held_from);
      subs = p.H_k * p.blocks;
    }
    tiles = tiles_of(length);
  }
  __device__ __forceinline__ void next(const AttentionParams& p, int lane) {
    if (++t < tiles) return;
    t = 0;
    if (++sub < subs) return;
    sub = 0;
    ++n;
    while (n < p.N) {  // to the next sequence with keys
      if (n - held_from >= 32) hold(p, lane);
      const unsigned some = __ballot_sync(0xffffffffu, held > 0) >> (n - held_from);
      if (some) {
        n += __ffs(some) - 1;
        break;
      }
      n = held_from + 32;
    }
    if (n > p.N) n = p.N;
    enter(p, lane);
  }
};

// 16 bytes to shared memory, zeros where there is nothing to copy.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(some ? 16 : 0) : "memory");
}
// Arrives (as one of those that the barrier counts) once this thread's copies so far are there.
__device__ __forceinline__ void arrive_copied(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The rows of a unit.
struct Unit {
  int tok0, head0, r0, rows;
  __device__ __forceinline__ Unit(const AttentionParams& p, const Walk& w) {
    const bool own = w.n < p.N;
    const int blocks = own ? p.blocks : p.prefix_blocks, head = w.sub / blocks;
    head0 = head * p.group;
    r0 = (w.sub - head * blocks) * kRows;
    tok0 = own ? w.n * p.tokens : 0;
    rows = min(kRows, (own ? p.tokens : p.N * p.tokens) * p.group - r0);
  }
};

// The copying warp.
__device__ __forceinline__ void copy_tiles(const AttentionParams& p, uint8_t* smem, Bars& bar, Walk walk, int count, uint64_t limit) {
  const int lane = threadIdx.x & 31, boxes = kTile / p.box_rows;
  const auto page_of = [&](const Walk& w) -> int64_t {  // of the lane's box: -2 behind the length, -1 outside the cache
    const int key = w.t * kTile + lane * p.box_rows;
    if (lane >= boxes || key >= w.length) return -2;
    const int64_t page = w.n < p.N ? index_at(p.table, p.table_dtype, w.n * p.table_st + key / p.page_size)
                                   : index_at(p.prefix_pages, p.prefix_dtype, key / p.page_size);
    return page < 0 || page >= p.pages ? -1 : page;
  };
  int64_t page = page_of(walk);
  int issued = 0;
  for (int k = 0; k < count; ++k) {
    const int stage = k % kStages;
    Walk ahead = walk;
    int64_t page_ahead = -2;
    if (k + 1 < count) {
      ahead.next(p, lane);
      page_ahead = page_of(ahead);
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&bar.empty[stage], (k / kStages + 1) & 1, limit))) {
      if (lane == 0) atomicOr(p.dev_err, kDevErrTimeout);
      break;
    }
    ++issued;
    const bool bad = __any_sync(0xffffffffu, page == -1), held = p.hold_copies && k == 0;
    const unsigned some = __ballot_sync(0xffffffffu, page >= 0);
    uint8_t* tile = smem + stage * kTileBytes;
    uint64_t* full = &bar.full[stage];
    if (lane == 0) {
      bar.bad[stage] = bad;
      if (bad) atomicOr(p.dev_err, kDevErrPage);
      mbar_arrive_expect_tx(full, __popc(some) * p.box_rows * 512);
    }
    __syncwarp();
    if (page >= 0 && !held) {
      const int row = (walk.t * kTile + lane * p.box_rows) % p.page_size, head = walk.sub / (walk.n < p.N ? p.blocks : p.prefix_blocks);
      uint8_t* at = tile + lane * p.box_rows * 128;
      for (int half = 0; half < 2; ++half) {
        tma_load_4d(at + half * kHalfBytes, &p.tm_k, full, 64 * half, head, row, (int)page);
        tma_load_4d(at + (2 + half) * kHalfBytes, &p.tm_v, full, 64 * half, head, row, (int)page);
      }
    }
    if (k == 0 || walk.t == 0) {  // the queries: half a warp a row
      const Unit u(p, walk);
      const uint32_t to = smem_u32(smem + kStages * kTileBytes + stage * kQueryBytes);
      const int chunk = lane & 15;
#pragma unroll
      for (int j = 0; j < kRows / 2; ++j) {
        const int i = 2 * j + (lane >> 4), r = u.r0 + i;
        const bool some_row = i < u.rows;
        const uint16_t* from = reinterpret_cast<const uint16_t*>(p.q);
        if (some_row) from += (int64_t)(u.tok0 + r / p.group) * p.q_st + (int64_t)(u.head0 + r % p.group) * p.q_sh + 8 * chunk;
        copy16(to + i * 256 + ((chunk ^ (i & 7)) << 4), from, some_row);
      }
      arrive_copied(full);
    } else {
      mbar_arrive(full);
    }
    walk = ahead;
    page = page_ahead;
  }
  // every copy ends before the memory is another's
  for (int k = max(0, issued - kStages); k < issued; ++k)
    if (!(p.hold_copies && k == 0)) mbar_wait(&bar.full[k % kStages], (k / kStages) & 1, kWaitNs);
}

template <bool F16>
__global__ void __launch_bounds__(kThreads, kResident) gdn_attention_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bar = *reinterpret_cast<Bars*>(smem + kStages * (kTileBytes + kQueryBytes));
  if (smem_u32(smem) & 1023) {  // where the swizzled tiles have to be; two workers would not fit an SM with room to spare for it
    if (threadIdx.x == 0) atomicOr(p.dev_err, kDevErrTimeout);
    grid_wait();
    return;
  }
  go_ahead();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.full[i], 33);     // the copying warp's lanes, and one of them for the tensor copies
      mbar_init(&bar.empty[i], kWarps);
    }
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  // Each thread of the first four warps counts the tiles of N / 128 sequences in a row, then the threads' sums are joined.
  constexpr int kCounting = 32 * kWarps;
  const int subs = p.H_k * p.blocks, each = (p.N + kCounting - 1) / kCounting;
  const int64_t prefix_tiles = (int64_t)tiles_of(p.prefix) * p.H_k * p.prefix_blocks;
  int64_t total, sharers;
  {
    int64_t mine = 0, before = 0;
    bool bad = false;
    if (warp < kWarps)
      for (int i = 0, n = tid * each; i < each && n < p.N; ++i, ++n) {
        const int length = length_of(p, n);
        bad |= length < 0;
        mine += tiles_of(length);
      }
    if (bad && blockIdx.x == 0) atomicOr(p.dev_err, kDevErrLength);
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
    if (lane == 31) bar.found[warp] = upto;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += bar.found[w];
      all += bar.found[w];
    }
    before += upto - mine;
    total = all * subs + prefix_tiles;
    __syncthreads();
    // no more workers than tiles: one without any between two parts of a unit would leave a gap
    sharers = total < gridDim.x ? total : (int64_t)gridDim.x;
    if (blockIdx.x >= sharers) {
      grid_wait();
      return;
    }
    const int64_t a = total * blockIdx.x / sharers;
    if (warp < kWarps && before * subs <= a && a < (before + mine) * subs) {  // the share begins in one of these
      int64_t at = before;
      for (int i = 0, n = tid * each; i < each && n < p.N; ++i, ++n) {
        const int tiles = tiles_of(length_of(p, n));
        if (a < (at + tiles) * subs) {
          const int64_t in = a - at * subs;
          bar.found[0] = n;
          bar.found[1] = in / tiles;
          bar.found[2] = in % tiles;
          break;
        }
        at += tiles;
      }
    }
    if (tid == 0 && a >= all * subs && prefix_tiles) {
      const int64_t in = a - all * subs, tiles = tiles_of(p.prefix);
      bar.found[0] = p.N;
      bar.found[1] = in / tiles;
      bar.found[2] = in % tiles;
    }
    __syncthreads();
  }
  const int count = (int)(total * (blockIdx.x + 1) / sharers - total * blockIdx.x / sharers);  // at least one
  Walk take;
  take.n = (int)bar.found[0];
  take.sub = (int)bar.found[1];
  take.t = (int)bar.found[2];
  take.hold(p, lane);
  take.enter(p, lane);
  const uint64_t limit = p.wait_ns ? p.wait_ns : kWaitNs;
  if (warp == kWarps) {
    copy_tiles(p, smem, bar, take, count, limit);
    return;
  }

  // All four warps walk the same units whatever happens on the way, so that they meet at the same ends.
  const float c = fabsf(p.scale) * kLog2e;
  const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
  constexpr float kBias = F16 ? 6.f : 0.f;  // f16 weights are kept 2^6 above their normal range's end for longer
  const int mi = lane >> 3, mj = lane & 7;
  uint32_t q[8][4];
  float base[2], sum[2], o[16][4];
  bool starts = false, unit_bad = false, dead = false;
#pragma unroll 1
  for (int k = 0; k < count; ++k) {
    const int stage = k % kStages;
    uint8_t* tile = smem + stage * kTileBytes;
    if (!dead && !__all_sync(0xffffffffu, mbar_wait(&bar.full[stage], (k / kStages) & 1, limit))) {
      dead = true;
      if (lane == 0) atomicOr(p.dev_err, kDevErrTimeout);
    }
    const Unit u(p, take);
    const bool own = take.n < p.N;
    if (k == 0 || take.t == 0) {
      starts = take.t == 0;
      unit_bad = false;
      const uint32_t at = smem_u32(smem + kStages * kTileBytes + stage * kQueryBytes) + ((mi & 1) * 8 + mj) * 256;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        ldmatrix_x4(at + (((2 * kk + (mi >> 1)) ^ mj) << 4), q[kk]);
#pragma unroll
        for (int e = 0; e < 4; ++e) q[kk][e] ^= flip;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        base[i] = -INFINITY;
        sum[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    }
    unit_bad |= dead || bar.bad[stage];
    const int key0 = take.t * kTile + warp * kWarpKeys, valid = min(kWarpKeys, take.length - key0);
    if (valid > 0 && !unit_bad) {
      const uint32_t kb = smem_u32(tile) + warp * kWarpKeys * 128, vb = kb + 2 * kHalfBytes;
      float acc[2][2][4] = {};  // [even and odd steps][keys]
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int key = (mi >> 1) * 8 + mj, chunk = 2 * kk + (mi & 1);
        uint32_t b[4];
        ldmatrix_x4(kb + (chunk >> 3) * kHalfBytes + key * 128 + (((chunk & 7) ^ (key & 7)) << 4), b);
        mma16<F16>(acc[kk & 1][0], q[kk], b[0], b[1]);
        mma16<F16>(acc[kk & 1][1], q[kk], b[2], b[3]);
      }
      float w[2][4];
      const int tail = own && p.tokens > 1 ? max(0, take.length - p.tokens + 1) : take.length;  // keys from here on are not for all rows
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[h][e] = (acc[0][h][e] + acc[1][h][e]) * c;
      if (key0 + kWarpKeys > tail) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + 8 * h + 2 * (lane & 3) + (e & 1), r = u.r0 + lane / 4 + 8 * (e >> 1);
            const int seen = own ? take.length - p.tokens + 1 + r / p.group : take.length;
            if (key >= min(seen, take.length)) w[h][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], w[h][e]);
      bool moves = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        moves |= top[i] > base[i] + (kRoom + kBias);
      }
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float now = fmaxf(base[i], top[i] - kBias);
          const float keep = now == -INFINITY || now == base[i] ? 1.f : exp2_fast(base[i] - now);
          base[i] = now;
          sum[i] *= keep;
#pragma unroll
          for (int j = 0; j < 16; ++j) { o[j][2 * i] *= keep; o[j][2 * i + 1] *= keep; }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float from_base = base[i] == -INFINITY ? 0.f : base[i];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 2 * i; e < 2 * i + 2; ++e) {
            w[h][e] = exp2_fast(w[h][e] - from_base);
            sum[i] += w[h][e];
          }
      }
      const int clean = min(valid, max(0, tail - key0));  // keys that all rows see
      if (clean < kWarpKeys) {
        // What lies behind must not meet the products, be its weight zero: an infinity would leave a NaN.
        // Keys that some rows see are added by hand, the places are cleared.
#pragma unroll 1
        for (int j = clean; j < valid; ++j) {
          const int from = (lane & ~3) | ((j & 7) >> 1);
          float pj[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x0 = j < 8 ? w[0][2 * i] : w[1][2 * i], x1 = j < 8 ? w[0][2 * i + 1] : w[1][2 * i + 1];
            pj[i] = __shfl_sync(0xffffffffu, j & 1 ? x1 : x0, from);
            const int r = u.r0 + lane / 4 + 8 * i;
            if (key0 + j >= take.length - p.tokens + 1 + r / p.group) pj[i] = -1.f;  // not seen
          }
#pragma unroll
          for (int nt = 0; nt < 16; ++nt) {
            uint32_t x;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(vb + (nt >> 3) * kHalfBytes + j * 128 + (((nt & 7) ^ (j & 7)) << 4) + 4 * (lane & 3)));
            const float2 v = unpack16<F16>(x);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (pj[i] >= 0.f || pj[i] != pj[i]) {
                o[nt][2 * i] = fmaf(pj[i], v.x, o[nt][2 * i]);
                o[nt][2 * i + 1] = fmaf(pj[i], v.y, o[nt][2 * i + 1]);
              }
            }
          }
        }
        __syncwarp();
        for (int i = lane; i < (kWarpKeys - clean) * 16; i += 32) {
          const int j = clean + i / 16, chunk = i % 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (chunk >> 3) * kHalfBytes + j * 128 + ((chunk & 7) << 4)), "r"(0) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * h + 2 * (lane & 3) + (e & 1) >= clean) w[h][e] = 0.f;
      }
      const uint32_t a[4] = {pack16x2<F16>(w[0][0], w[0][1]), pack16x2<F16>(w[0][2], w[0][3]), pack16x2<F16>(w[1][0], w[1][1]),
                             pack16x2<F16>(w[1][2], w[1][3])};
#pragma unroll
      for (int nt = 0; nt < 16; nt += 2) {
        const int key = (mi & 1) * 8 + mj, chunk = nt + (mi >> 1);
        uint32_t b[4];
        ldmatrix_x4_trans(vb + (chunk >> 3) * kHalfBytes + key * 128 + (((chunk & 7) ^ (key & 7)) << 4), b);
        mma16<F16>(o[nt], a, b[0], b[1]);
        mma16<F16>(o[nt + 1], a, b[2], b[3]);
      }
    }
    const bool ends = take.t + 1 == take.tiles;
    if (ends || k + 1 == count) {  // the warps' parts of the unit come together, over the tile
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        if ((lane & 3) == 0) bar.ml[warp][lane / 4 + 8 * i] = make_float2(base[i], unit_bad ? kBad : sum[i]);
      }
      float* join = reinterpret_cast<float*>(tile);   // [warp][16][128], columns by eights turned by the row
      named_sync(1, 32 * kWarps);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int at = lane / 4 + 8 * i;
          *reinterpret_cast<float2*>(join + (warp * kRows + at) * kHeadDim + ((j ^ (at & 7)) * 8 + 2 * (lane & 3))) =
              make_float2(o[j][2 * i], o[j][2 * i + 1]);
        }
      named_sync(1, 32 * kWarps);
      const int unit = take.n * subs + take.sub, worker = (int)blockIdx.x;
      const bool whole = starts && ends;
      if (tid == 0) {
        if (starts) p.first_worker[unit] = worker;
        if (ends) p.last_worker[unit] = worker;
      }
      const int64_t slot = whole ? 2 * p.workers + (int64_t)unit : 2 * worker + (starts ? 1 : 0);
      const int cg = tid & 15;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = tid / 16 + 8 * i, r = u.r0 + row;
        if (row >= u.rows) break;
        float2 ml[kWarps];
        float top = -INFINITY, l = 0.f, x[8] = {};
        bool bad = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          ml[w] = bar.ml[w][row];
          top = fmaxf(top, ml[w].x);
          bad |= ml[w].y == kBad;
        }
        const float from_base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = exp2_fast(ml[w].x - from_base);
          const float4* y = reinterpret_cast<const float4*>(join + (w * kRows + row) * kHeadDim + (cg ^ (row & 7)) * 8);
          const float4 y0 = y[0], y1 = y[1];
          l = fmaf(f, ml[w].y, l);
          x[0] = fmaf(f, y0.x, x[0]); x[1] = fmaf(f, y0.y, x[1]); x[2] = fmaf(f, y0.z, x[2]); x[3] = fmaf(f, y0.w, x[3]);
          x[4] = fmaf(f, y1.x, x[4]); x[5] = fmaf(f, y1.y, x[5]); x[6] = fmaf(f, y1.z, x[6]); x[7] = fmaf(f, y1.w, x[7]);
        }
        if (whole && !p.prefix) {
          if (!bad) {
            const float inv = top == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inv;
            const int64_t token = u.tok0 + r / p.group;
            const int head = u.head0 + r % p.group;
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + token * p.o_st + head * p.o_sh + 8 * cg) = pack16x8<F16>(x);
            if (p.lse && cg == 0)
              p.lse[token * p.lse_st + head] = top == -INFINITY && l == 0.f ? -INFINITY : (from_base + log2f(l)) * kLn2;
          }
        } else {
          float4* y = reinterpret_cast<float4*>(p.part_o + (slot * p.block_rows + row) * kHeadDim + 8 * cg);
          y[0] = make_float4(x[0], x[1], x[2], x[3]);
          y[1] = make_float4(x[4], x[5], x[6], x[7]);
          if (cg == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * p.block_rows + row) * 2) = make_float2(top, bad ? kBad : l);
        }
      }
      fence_proxy_async_smem();
      named_sync(1, 32 * kWarps);   // the sums before the next unit's, too
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.empty[stage]);
    if (k + 1 < count) take.next(p, lane);
  }
  grid_wait();
}

// The parts of the units that were cut, and those of the prefix: `kPer` warps for each row take turns at its
// parts, four on their way at a time, lanes four columns each.
template <bool F16, int kPer>
__global__ void __launch_bounds__(kPer > 4 ? 32 * kPer : 128) gdn_attention_join_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kRowsHere = kPer >= 4 ? 1 : 4 / kPer;
  __shared__ float s_o[kPer][kHeadDim];
  __shared__ float2 s_ml[kPer];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5 & (kPer - 1);
  const int64_t id = (int64_t)blockIdx.x * kRowsHere + (kPer >= 4 ? 0 : threadIdx.x >> 5);
  grid_wait();
  if (id >= (int64_t)p.N * p.H_k * p.blocks * p.block_rows) return;
  const int unit = (int)(id / p.block_rows), row = (int)(id - (int64_t)unit * p.block_rows);
  const int subs = p.H_k * p.blocks, n = unit / subs, sub = unit - n * subs, hk = sub / p.blocks;
  const int r = (sub - hk * p.blocks) * kRows + row;
  if (r >= p.tokens * p.group) return;
  const int length = length_of(p, n);
  // the sequence's own parts: of worker `first` and those behind it, or one of a whole unit
  int first = p.first_worker[unit], own = p.last_worker[unit] - first + 1;
  if (length <= 0) first = own = 0;
  // the prefix' parts of the row, of this kind's workers or of those of the prefix kernel
  int prefix_first = 0, shared = 0, prefix_unit = 0;
  const int pr = n * p.tokens * p.group + r;
  const bool many = p.prefix_units > 0;
  int turns = 1;  // sums of the row that a worker of the prefix kernel has
  if (many) {
    prefix_unit = hk * p.prefix_units + pr / kPrefixRows;
    const int64_t tiles = (p.prefix + kPrefixKeys - 1) / kPrefixKeys, total = tiles * p.H_k * p.prefix_units, at = prefix_unit * tiles;
    prefix_first = (int)(((at + 1) * p.prefix_workers - 1) / total);   // the worker whose share holds tile `at`
    shared = (int)(((at + tiles) * p.prefix_workers - 1) / total) - prefix_first + 1;
    turns = p.N * p.tokens * p.group - pr / kPrefixRows * kPrefixRows <= 128 ? 2 : 1;
  } else if (p.prefix) {
    prefix_unit = p.N * subs + hk * p.prefix_blocks + pr / kRows;
    prefix_first = p.first_worker[prefix_unit];
    shared = p.last_worker[prefix_unit] - prefix_first + 1;
  }
  if (length < 0 || (own == 1 && !p.prefix)) return;  // none, or it is in the output
  // parts of no worker: the kernel before this one gave up, and said so
  bool bad = first < 0 || own < 0 || first + own > p.workers || prefix_first < 0 || shared < 0 ||
             prefix_first + shared > (many ? p.prefix_workers : p.workers);
  if (bad) own = shared = 0;
  const int parts_all = own + shared * turns;
  float top = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < parts_all; i0 += 4 * kPer) {
    float2 ml[4];
    float4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e * kPer;
      const bool of_prefix = i >= own, of_many = of_prefix && many;
      const int j2 = of_prefix ? i - own : i, j = of_prefix && turns == 2 ? j2 >> 1 : j2, turn = of_prefix && turns == 2 ? j2 & 1 : 0;
      const int parts = of_prefix ? shared : own, w = (of_prefix ? prefix_first : first) + j;
      const int workers = of_many ? p.prefix_workers : p.workers;
      const int64_t slot = parts == 1 ? 2 * (int64_t)workers + (of_prefix ? prefix_unit : unit) : 2 * w + (j == 0 ? 1 : 0);
      const int64_t at = of_many ? slot * kPrefixRows + pr % kPrefixRows + 128 * turn : slot * p.block_rows + (of_prefix ? pr % kRows : row);
      ml[e] = make_float2(-INFINITY, 0.f);
      x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < parts_all) {
        ml[e] = *reinterpret_cast<const float2*>((of_many ? p.prefix_ml : p.part_ml) + 2 * at);
        const float* y = of_many ? p.prefix_o + (slot * kHeadDim + lane / 2 * 8) * kPrefixRows + (pr % kPrefixRows + 128 * turn) * 8 + (lane & 1) * 4
                                 : p.part_o + at * kHeadDim + 4 * lane;
        x[e] = *reinterpret_cast<const float4*>(y);
        if (ml[e].y == 0.f) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);  // no key: nothing was written
      }
    }
    float now = top;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      now = fmaxf(now, ml[e].x);
      bad |= ml[e].y == kBad;
    }
    const float from_base = now == -INFINITY ? 0.f : now, keep = exp2_fast(top - from_base);
    top = now;
    l *= keep;
    o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float f = exp2_fast(ml[e].x - from_base);
      l = fmaf(f, ml[e].y, l);
      o = make_float4(fmaf(f, x[e].x, o.x), fmaf(f, x[e].y, o.y), fmaf(f, x[e].z, o.z), fmaf(f, x[e].w, o.w));
    }
  }
  if constexpr (kPer > 1) {
    reinterpret_cast<float4*>(s_o[warp])[lane] = o;
    if (lane == 0) s_ml[warp] = make_float2(top, l);
    bad = __syncthreads_or(bad);
    if (warp > 0) return;
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kPer; ++w) top = fmaxf(top, s_ml[w].x);
    const float from_base = top == -INFINITY ? 0.f : top;
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kPer; ++w) {
      const float f = exp2_fast(s_ml[w].x - from_base);
      const float4 x = reinterpret_cast<const float4*>(s_o[w])[lane];
      l = fmaf(f, s_ml[w].y, l);
      o = make_float4(fmaf(f, x.x, o.x), fmaf(f, x.y, o.y), fmaf(f, x.z, o.z), fmaf(f, x.w, o.w));
    }
  }
  if (bad) return;
  const float from_base = top == -INFINITY ? 0.f : top;
  const bool none = top == -INFINITY && l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  const int64_t token = n * (int64_t)p.tokens + r / p.group;
  const int head = hk * p.group + r % p.group;
  *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + token * p.o_st + head * p.o_sh + 4 * lane) =
      make_uint2(pack16x2<F16>(o.x * inv, o.y * inv), pack16x2<F16>(o.z * inv, o.w * inv));
  if (p.lse && lane == 0) p.lse[token * p.lse_st + head] = none ? -INFINITY : (from_base + log2f(l)) * kLn2;
}

// A kernel that may start before the one in front of it has ended (it waits for it itself).
template <typename Kernel>
cudaError_t launch_behind(Kernel kernel, int64_t grid, int threads, int smem, bool behind, const AttentionParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, p);
}

template <bool F16>
cudaError_t launch(const AttentionParams& p, cudaStream_t stream) {
  static thread_local int generation = -1, device = -1;  // the attribute is one of a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (generation != launch_config_generation() || device != dev) {
    e = cudaFuncSetAttribute(gdn_attention_kernel<F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    generation = launch_config_generation();
    device = dev;
  }
  const int64_t subs = (int64_t)p.H_k * p.blocks, own_units = p.N * subs;
  const int64_t most = ((int64_t)p.max_pages * p.page_size + kTile - 1) / kTile * own_units +
                       ((int64_t)p.prefix + kTile - 1) / kTile * p.H_k * p.prefix_blocks;
  const bool many = p.prefix_units > 0;
  if (many && (e = launch_attention_prefix(p, stream)) != cudaSuccess) return e;
  if (most) {
    e = launch_behind(gdn_attention_kernel<F16>, std::min<int64_t>(p.workers, most), kThreads, kSmemBytes, many, p, stream);
    if (e != cudaSuccess) return e;
  }
  // Warps a row by the parts that a row has about: 16 rows of 152 parts each take 5 us with sixteen, 26 with four.
  int64_t parts = 1 + p.workers / (own_units + p.H_k * p.prefix_blocks);
  if (many) parts += 1 + p.prefix_workers / ((int64_t)p.H_k * p.prefix_units);
  const int64_t rows = own_units * p.block_rows;
  if (parts <= 8) return launch_behind(gdn_attention_join_kernel<F16, 1>, (rows + 3) / 4, 128, 0, true, p, stream);
  if (parts <= 32) return launch_behind(gdn_attention_join_kernel<F16, 4>, rows, 128, 0, true, p, stream);
  return launch_behind(gdn_attention_join_kernel<F16, 16>, rows, 512, 0, true, p, stream);
}

}  // namespace

size_t plan_attention(AttentionParams* p, int sms, void* workspace) {
  p->group = p->H_q / p->H_k;
  const int64_t rows = (int64_t)p->tokens * p->group, all = p->N * rows;
  const bool many = p->prefix && all > kRows;
  p->workers = kResident * sms;
  p->blocks = (int32_t)((rows + kRows - 1) / kRows);
  p->prefix_blocks = p->prefix && !many ? 1 : 0;
  p->block_rows = (int32_t)std::min<int64_t>(kRows, p->prefix_blocks ? all : rows);
  p->prefix_units = many ? (int32_t)((all + kPrefixRows - 1) / kPrefixRows) : 0;
  const int64_t many_units = (int64_t)p->H_k * p->prefix_units;
  p->prefix_workers = many ? (int32_t)std::min<int64_t>(sms, many_units * (((int64_t)p->prefix + kPrefixKeys - 1) / kPrefixKeys)) : 0;
  const int64_t units = (int64_t)p->N * p->H_k * p->blocks + (int64_t)p->H_k * p->prefix_blocks;
  const int64_t slots = (2 * (int64_t)p->workers + (p->prefix ? units : 0)) * p->block_rows;
  const int64_t many_slots = many ? (2 * (int64_t)sms + many_units) * kPrefixRows : 0;
  size_t end = 0;
  auto take = [&](size_t bytes) {
    char* at = static_cast<char*>(workspace) + end;
    end += (bytes + 255) / 256 * 256;
    return at;
  };
  float* part_o = reinterpret_cast<float*>(take((size_t)slots * kHeadDim * 4));
  float* prefix_o = reinterpret_cast<float*>(take((size_t)many_slots * kHeadDim * 4));
  float* part_ml = reinterpret_cast<float*>(take((size_t)slots * 8));
  float* prefix_ml = reinterpret_cast<float*>(take((size_t)many_slots * 8));
  int32_t* first_worker = reinterpret_cast<int32_t*>(take((size_t)units * 8));
  if (workspace) {
    p->part_o = part_o; p->part_ml = part_ml;
    p->prefix_o = prefix_o; p->prefix_ml = prefix_ml;
    p->first_worker = first_worker; p->last_worker = first_worker + units;
  }
  return end;
}

cudaError_t launch_attention(const AttentionParams& p, cudaStream_t stream) {
  return p.op_f16 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace gdn
