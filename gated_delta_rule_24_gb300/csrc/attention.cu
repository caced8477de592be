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
// HBM bandwidth as long as copies are always under way.  Each of a worker's four warps takes 16 of a tile's
// keys on its own: a ring of tensor copies (box_rows places of a page each) that it issues and waits for
// itself, scores and sums by warp products with the keys as the narrow side, weights passed on in
// registers.  The warps meet at the end of a unit only.
#include <cuda_runtime.h>

#include <algorithm>

#include "attention.h"
#include "decay.cuh"
#include "ptx.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kWarpKeys = 16, kTile = kWarps * kWarpKeys;
constexpr int kRows = 16;                      // rows of a unit
constexpr int kStages = 3;
constexpr int kHalfBytes = kWarpKeys * 128;    // 64 of a row's 128 values
constexpr int kStageBytes = 4 * kHalfBytes;    // keys, then values
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kJoinBytes = kWarps * kRows * 64 * 4;   // half the columns of every warp's sums
constexpr int kSmemBytes = kRingBytes + kJoinBytes + kWarps * kRows * 8 + kWarps * kStages * 8 + 64;
constexpr int kResident = 2;                   // workers on an SM
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
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

struct Smem {
  uint8_t* ring;   // [warp][stage]
  float* join;     // [warp][16][64], columns by eights turned by the row
  float2* ml;      // [warp][16]
  uint64_t* full;  // [warp][stage]
  int64_t* found;  // the walk's start
};

template <bool F16>
__global__ void __launch_bounds__(kThreads, kResident) gdn_attention_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem s;
  s.ring = raw;
  if (smem_u32(raw) & 1023) {  // where the swizzled tiles have to be; two workers would not fit an SM with room to spare for it
    if (threadIdx.x == 0) atomicOr(p.dev_err, kDevErrTimeout);
    return;
  }
  s.join = reinterpret_cast<float*>(s.ring + kRingBytes);
  s.ml = reinterpret_cast<float2*>(s.ring + kRingBytes + kJoinBytes);
  s.full = reinterpret_cast<uint64_t*>(s.ml + kWarps * kRows);
  s.found = reinterpret_cast<int64_t*>(s.full + kWarps * kStages);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* full = s.full + warp * kStages;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  // Each thread counts the tiles of N / 128 sequences in a row, then the threads' sums are joined.
  const int subs = p.H_k * p.blocks, each = (p.N + kThreads - 1) / kThreads;
  const int64_t prefix_tiles = (int64_t)tiles_of(p.prefix) * p.H_k * p.prefix_blocks;
  int64_t before = 0, total, sharers;
  {
    int64_t mine = 0;
    bool bad = false;
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
    if (lane == 31) s.found[warp] = upto;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s.found[w];
      all += s.found[w];
    }
    before += upto - mine;
    total = all * subs + prefix_tiles;
    __syncthreads();
    // no more workers than tiles: one without any between two parts of a unit would leave a gap
    sharers = total < gridDim.x ? total : (int64_t)gridDim.x;
    if (blockIdx.x >= sharers) return;
    const int64_t a = total * blockIdx.x / sharers;
    if (before * subs <= a && a < (before + mine) * subs) {  // the share begins in one of these
      int64_t at = before;
      for (int i = 0, n = tid * each; i < each && n < p.N; ++i, ++n) {
        const int tiles = tiles_of(length_of(p, n));
        if (a < (at + tiles) * subs) {
          const int64_t in = a - at * subs;
          s.found[0] = n;
          s.found[1] = in / tiles;
          s.found[2] = in % tiles;
          break;
        }
        at += tiles;
      }
    }
    if (tid == 0 && a >= all * subs && prefix_tiles) {
      const int64_t in = a - all * subs, tiles = tiles_of(p.prefix);
      s.found[0] = p.N;
      s.found[1] = in / tiles;
      s.found[2] = in % tiles;
    }
    __syncthreads();
  }
  const int count = (int)(total * (blockIdx.x + 1) / sharers - total * blockIdx.x / sharers);  // at least one
  Walk take, load;
  take.n = (int)s.found[0];
  take.sub = (int)s.found[1];
  take.t = (int)s.found[2];
  take.hold(p, lane);
  take.enter(p, lane);
  load = take;

  const uint64_t limit = p.wait_ns ? p.wait_ns : 200000000ull;
  uint8_t* ring = s.ring + warp * kStages * kStageBytes;
  int dead_at = count;      // the tile whose wait ran out: from there on no more copies, no more waits
  bool dead = false;
  uint32_t bad_stage = 0;   // stages whose tile has a bad page
  const int boxes = kWarpKeys / p.box_rows;
  int64_t held_pages = -1;
  int held_n = -1, held_box = 0;   // lane i holds the page of the warp's box held_box + i of sequence held_n
  auto issue = [&](int k) {
    const int stage = k % kStages;
    const int box0 = load.t * boxes;
    if (load.n != held_n || box0 < held_box || box0 + boxes > held_box + 32) {
      held_n = load.n;
      held_box = box0;
      const int box = box0 + lane, key = box / boxes * kTile + warp * kWarpKeys + box % boxes * p.box_rows;
      held_pages = -1;
      if (key < load.length) {
        held_pages = load.n < p.N ? index_at(p.table, p.table_dtype, load.n * p.table_st + key / p.page_size)
                                  : index_at(p.prefix_pages, p.prefix_dtype, key / p.page_size);
      }
    }
    const int head = load.sub / (load.n < p.N ? p.blocks : p.prefix_blocks);
    uint8_t* at = ring + stage * kStageBytes;
    int copies = 0;
    bool bad = false;
    int64_t page[2];
    int row[2];
    for (int i = 0; i < boxes; ++i) {
      const int key = load.t * kTile + warp * kWarpKeys + i * p.box_rows;
      page[i] = __shfl_sync(0xffffffffu, held_pages, box0 - held_box + i);
      row[i] = key % p.page_size;
      if (key < load.length) {
        if (page[i] < 0 || page[i] >= p.pages) { bad = true; page[i] = -1; }
        else ++copies;
      } else {
        page[i] = -1;
      }
    }
    if (bad) {
      bad_stage |= 1u << stage;
      if (lane == 0) atomicOr(p.dev_err, kDevErrPage);
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[stage], copies * 4 * p.box_rows * 128);
      if (!(p.hold_copies && k == 0)) {
        for (int i = 0; i < boxes; ++i) {
          if (page[i] < 0) continue;
          for (int half = 0; half < 2; ++half) {
            tma_load_4d(at + half * kHalfBytes + i * 1024, &p.tm_k, &full[stage], 64 * half, head, row[i], (int)page[i]);
            tma_load_4d(at + (2 + half) * kHalfBytes + i * 1024, &p.tm_v, &full[stage], 64 * half, head, row[i], (int)page[i]);
          }
        }
      }
    }
    load.next(p, lane);
  };
  for (int k = 0; k < min(count, kStages); ++k) issue(k);

  const float c = fabsf(p.scale) * kLog2e;
  const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
  constexpr float kBias = F16 ? 6.f : 0.f;  // f16 weights are kept 2^6 above their normal range's end for longer
  uint32_t q[8][4];
  float base[2], sum[2], o[16][4];
  bool starts = false, unit_bad = false;
  int rows = 0, tok0 = 0, r0 = 0, head0 = 0;
#pragma unroll 1
  for (int k = 0; k < count; ++k) {
    const int stage = k % kStages;
    if (k == 0 || take.t == 0) {  // a unit
      starts = take.t == 0;
      unit_bad = false;
      const bool own = take.n < p.N;
      const int blocks = own ? p.blocks : p.prefix_blocks;
      head0 = take.sub / blocks * p.group;
      r0 = take.sub % blocks * kRows;
      tok0 = own ? take.n * p.tokens : 0;
      rows = (own ? p.tokens : p.N * p.tokens) * p.group;
      rows = min(kRows, rows - r0);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = lane / 4 + 8 * half, r = r0 + i;
        const uint16_t* row = reinterpret_cast<const uint16_t*>(p.q) + (int64_t)(tok0 + r / p.group) * p.q_st +
                              (int64_t)(head0 + r % p.group) * p.q_sh + 2 * (lane & 3);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          q[kk][half] = i < rows ? *reinterpret_cast<const uint32_t*>(row + 16 * kk) ^ flip : 0u;
          q[kk][half + 2] = i < rows ? *reinterpret_cast<const uint32_t*>(row + 16 * kk + 8) ^ flip : 0u;
        }
        base[half] = -INFINITY;
        sum[half] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    }
    if (!dead && !__all_sync(0xffffffffu, mbar_wait(&full[stage], (k / kStages) & 1, limit))) {
      dead = true;
      dead_at = k;
      if (lane == 0) atomicOr(p.dev_err, kDevErrTimeout);
    }
    unit_bad |= dead || (bad_stage >> stage & 1u);
    bad_stage &= ~(1u << stage);
    const int key0 = take.t * kTile + warp * kWarpKeys, valid = min(kWarpKeys, take.length - key0);
    if (valid > 0 && !unit_bad) {
      const uint32_t kb = smem_u32(ring + stage * kStageBytes), vb = kb + 2 * kHalfBytes;
      const int mi = lane >> 3, mj = lane & 7;
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
      const bool own = take.n < p.N;
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
            const int key = key0 + 8 * h + 2 * (lane & 3) + (e & 1), r = r0 + lane / 4 + 8 * (e >> 1);
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
            const int r = r0 + lane / 4 + 8 * i;
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
    __syncwarp();
    if (k + kStages < count && !dead) issue(k + kStages);
    const bool ends = take.t + 1 == take.tiles;
    if (ends || k + 1 == count) {  // the warps' parts of the unit come together, half the columns at a time
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        if ((lane & 3) == 0) s.ml[warp * kRows + lane / 4 + 8 * i] = make_float2(base[i], unit_bad ? kBad : sum[i]);
      }
      const int unit = take.n * subs + take.sub, worker = (int)blockIdx.x;
      const bool whole = starts && ends;
      if (tid == 0) {
        if (starts) p.first_worker[unit] = worker;
        if (ends) p.last_worker[unit] = worker;
      }
      const int64_t slot = whole ? 2 * p.workers + (int64_t)unit : 2 * worker + (starts ? 1 : 0);
      const int row = tid / 8, cg = tid % 8, r = r0 + row;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int at = lane / 4 + 8 * i;
            *reinterpret_cast<float2*>(s.join + (warp * kRows + at) * 64 + ((j ^ (at & 7)) * 8 + 2 * (lane & 3))) =
                make_float2(o[8 * half + j][2 * i], o[8 * half + j][2 * i + 1]);
          }
        __syncthreads();
        float2 ml[kWarps];
        float top = -INFINITY, l = 0.f, x[8] = {};
        bool bad = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          ml[w] = s.ml[w * kRows + row];
          top = fmaxf(top, ml[w].x);
          bad |= ml[w].y == kBad;
        }
        const float from_base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = exp2_fast(ml[w].x - from_base);
          const float4* y = reinterpret_cast<const float4*>(s.join + (w * kRows + row) * 64 + (cg ^ (row & 7)) * 8);
          const float4 y0 = y[0], y1 = y[1];
          l = fmaf(f, ml[w].y, l);
          x[0] = fmaf(f, y0.x, x[0]); x[1] = fmaf(f, y0.y, x[1]); x[2] = fmaf(f, y0.z, x[2]); x[3] = fmaf(f, y0.w, x[3]);
          x[4] = fmaf(f, y1.x, x[4]); x[5] = fmaf(f, y1.y, x[5]); x[6] = fmaf(f, y1.z, x[6]); x[7] = fmaf(f, y1.w, x[7]);
        }
        if (row < rows) {
          if (whole && !p.prefix) {
            if (!bad) {
              const float inv = top == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] *= inv;
              const int64_t token = tok0 + r / p.group;
              const int head = head0 + r % p.group;
              *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + token * p.o_st + head * p.o_sh + 64 * half + 8 * cg) = pack16x8<F16>(x);
              if (p.lse && half == 0 && cg == 0)
                p.lse[token * p.lse_st + head] = top == -INFINITY && l == 0.f ? -INFINITY : (from_base + log2f(l)) * kLn2;
            }
          } else {
            float4* y = reinterpret_cast<float4*>(p.part_o + (slot * p.block_rows + row) * kHeadDim + 64 * half + 8 * cg);
            y[0] = make_float4(x[0], x[1], x[2], x[3]);
            y[1] = make_float4(x[4], x[5], x[6], x[7]);
            if (half == 0 && cg == 0)
              *reinterpret_cast<float2*>(p.part_ml + (slot * p.block_rows + row) * 2) = make_float2(top, bad ? kBad : l);
          }
        }
        __syncthreads();
      }
    }
    if (k + 1 < count) take.next(p, lane);
  }
  // Copies that are still on their way after a wait ran out end before the memory is another's.
  for (int k = dead_at; k < min(count, dead_at + kStages); ++k)
    if (!(p.hold_copies && k == 0)) mbar_wait(&full[k % kStages], (k / kStages) & 1, 200000000ull);
}

// The parts of the units that were cut, and those of the prefix: one CTA for each row, its warps taking
// turns at the parts, lanes four columns each.
template <bool F16>
__global__ void __launch_bounds__(kThreads) gdn_attention_join_kernel(const __grid_constant__ AttentionParams p) {
  __shared__ float s_o[kWarps][kHeadDim];
  __shared__ float2 s_ml[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = (int)(blockIdx.x / (unsigned)p.block_rows), row = (int)(blockIdx.x % (unsigned)p.block_rows);
  const int subs = p.H_k * p.blocks, n = unit / subs, hk = unit % subs / p.blocks;
  const int r = unit % p.blocks * kRows + row;
  if (r >= p.tokens * p.group) return;
  const int length = length_of(p, n);
  if (length < 0) return;
  int first = 0, own = 0;  // the sequence's own parts: of worker `first` and those behind it, or one of a whole unit
  if (length > 0) {
    first = p.first_worker[unit];
    own = p.last_worker[unit] - first + 1;
  }
  if (own == 1 && !p.prefix) return;  // it is in the output
  // the prefix' parts of the row, of this kind's workers or of those of the prefix kernel
  int prefix_first = 0, shared = 0, prefix_unit = 0;
  const int pr = n * p.tokens * p.group + r;
  const bool many = p.prefix_units > 0;
  if (many) {
    prefix_unit = hk * p.prefix_units + pr / kPrefixRows;
    const int64_t tiles = (p.prefix + kPrefixKeys - 1) / kPrefixKeys, total = tiles * p.H_k * p.prefix_units, at = prefix_unit * tiles;
    prefix_first = (int)(((at + 1) * p.prefix_workers - 1) / total);   // the worker whose share holds tile `at`
    shared = (int)(((at + tiles) * p.prefix_workers - 1) / total) - prefix_first + 1;
  } else if (p.prefix) {
    prefix_unit = p.N * subs + hk * p.prefix_blocks + pr / kRows;
    prefix_first = p.first_worker[prefix_unit];
    shared = p.last_worker[prefix_unit] - prefix_first + 1;
  }
  float top = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // parts of no worker: the kernel before this one gave up, and said so
  bool bad = first < 0 || own < 0 || first + own > p.workers || prefix_first < 0 || shared < 0 ||
             prefix_first + shared > (many ? p.prefix_workers : p.workers);
  if (bad) own = shared = 0;
#pragma unroll 4
  for (int i = warp; i < own + shared; i += kWarps) {
    const bool of_prefix = i >= own;
    const int j = of_prefix ? i - own : i, parts = of_prefix ? shared : own, w = (of_prefix ? prefix_first : first) + j;
    const bool of_many = of_prefix && many;
    const int workers = of_many ? p.prefix_workers : p.workers;
    const int64_t slot = parts == 1 ? 2 * (int64_t)workers + (of_prefix ? prefix_unit : unit) : 2 * w + (j == 0 ? 1 : 0);
    const int64_t at = of_many ? slot * kPrefixRows + pr % kPrefixRows : slot * p.block_rows + (of_prefix ? pr % kRows : row);
    const float2 ml = *reinterpret_cast<const float2*>((of_many ? p.prefix_ml : p.part_ml) + 2 * at);
    const float4 x = *reinterpret_cast<const float4*>((of_many ? p.prefix_o : p.part_o) + at * kHeadDim + 4 * lane);
    bad |= ml.y == kBad;
    const float now = fmaxf(top, ml.x), from_base = now == -INFINITY ? 0.f : now;
    const float keep = exp2_fast(top - from_base), f = exp2_fast(ml.x - from_base);
    top = now;
    l = l * keep + f * ml.y;
    o = make_float4(o.x * keep + f * x.x, o.y * keep + f * x.y, o.z * keep + f * x.z, o.w * keep + f * x.w);
  }
  reinterpret_cast<float4*>(s_o[warp])[lane] = o;
  if (lane == 0) s_ml[warp] = make_float2(top, l);
  if (__syncthreads_or(bad)) return;
  float total = 0.f, x = 0.f;
  top = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w].x);
  const float from_base = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = exp2_fast(s_ml[w].x - from_base);
    total += f * s_ml[w].y;
    x += f * s_o[w][threadIdx.x];
  }
  const bool none = top == -INFINITY && total == 0.f;
  const int64_t token = n * (int64_t)p.tokens + r / p.group;
  const int head = hk * p.group + r % p.group;
  reinterpret_cast<uint16_t*>(p.out)[token * p.o_st + head * p.o_sh + threadIdx.x] = (uint16_t)pack16x2<F16>(none ? 0.f : x / total, 0.f);
  if (p.lse && threadIdx.x == 0) p.lse[token * p.lse_st + head] = none ? -INFINITY : (from_base + log2f(total)) * kLn2;
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
  const int64_t subs = (int64_t)p.H_k * p.blocks;
  const int64_t most = ((int64_t)p.max_pages * p.page_size + kTile - 1) / kTile * p.N * subs +
                       ((int64_t)p.prefix + kTile - 1) / kTile * p.H_k * p.prefix_blocks;
  if (p.prefix_units > 0 && (e = launch_attention_prefix(p, stream)) != cudaSuccess) return e;
  if (most) gdn_attention_kernel<F16><<<(unsigned)std::min<int64_t>(p.workers, most), kThreads, kSmemBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  gdn_attention_join_kernel<F16><<<(unsigned)(p.N * subs * p.block_rows), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
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
