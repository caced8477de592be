// The own pages of the sequences in the attention over a paged cache: what a worker does with its share
// (attention.cu says what workers, units and shares are).
//
// Each key and value is read once for up to 16 rows, 16 flops a byte at most (4 x 128 a row for 512 bytes): the kernel is bound by
// HBM bandwidth as long as copies are always under way.  A warp of its own looks up pages and issues the tensor
// copies (boxes of up to 64 places of a page) into a ring of three tiles, over the ends of units; with a unit's first
// tile come its queries.  Four warps take 16 of a tile's keys each: scores (keys x rows) and sums (values x rows) by warp
// products with eight rows, or two times eight, as the narrow side, so that few rows take few products and registers; weights
// are passed on in registers, in two parts of the values' type where that costs nothing.  The warps meet at the end of a unit only, over the memory of its last tile.
//
// Measured: 256 sequences of up to 8192 keys, 4.3 GB of pages in 634 us, 6.8 TB/s and as much as a copy; one sequence of
// 131072 keys, where no worker has more than some twenty tiles and the start and the join count, 27.6 us.
// A unit of 16 rows and one tile takes a worker 4.2 us, of 8 rows 3.0: four warps at a third of their issue slots, two workers an SM.
#pragma once
#include <type_traits>

#include "attention_common.cuh"

namespace gdn {
namespace own {

constexpr int kWarps = 4;                      // that compute; one more copies
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kWarpKeys = 16, kTile = kWarps * kWarpKeys;
static_assert(kTile == kOwnKeys, "boxes fit a tile");
constexpr int kRows = 16;                      // rows of a unit
constexpr int kStages = 3;
constexpr int kHeld = 512;                     // so many sequences' lengths are read once, when they are counted
constexpr int kKeysBytes = kTile * 256;
constexpr int kTileBytes = 2 * kKeysBytes;     // keys, then values; either box by box, a box' rows by halves of 64 values
constexpr int kQueryBytes = kRows * 256;
static_assert(kRows * kHeadDim * 4 == kWarpKeys * 512 && kRows * 256 == kWarpKeys * 256, "a warp's sums lie over its own keys and values");
// Where a share begins: tile t of `sub` of sequence n, after `index` tiles in all.
struct Place { uint32_t n, sub, t, index; };
struct Bars {
  float2 ml[2][kWarps][kRows];                 // of one piece, and of the next
  uint64_t full[kStages], empty[kStages], joined;
  Place found[2];                              // the share's ends
  uint32_t bad[kStages];                       // a page of the stage's tile is none
  int lengths[kHeld];
};
constexpr int kBytes = kStages * (kTileBytes + kQueryBytes) + sizeof(Bars);
constexpr int kPlace = (kBytes + 1023) / 1024 * 1024;   // of a worker beside another
__device__ __forceinline__ Bars& bars_of(uint8_t* smem) { return *reinterpret_cast<Bars*>(smem + kStages * (kTileBytes + kQueryBytes)); }
__device__ __forceinline__ int length_at(const AttentionParams& p, const Bars& bar, int n) { return n < kHeld ? bar.lengths[n] : length_of(p, n); }

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

// A value that the compiler takes for new here: what is made of it is not kept in registers from before, over loops that need them.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

__device__ __forceinline__ int tiles_of(int length) { return length > 0 ? (length + kTile - 1) / kTile : 0; }

// A tile of the walk through all units: sequence n (N: the prefix), `sub` = key head * groups of row blocks + group, tile t.  The
// blocks of a group are walked by as many workers side by side, so that a key that one reads is in L2 for the others.
// The lanes of a warp hold the lengths of 32 sequences.
struct Walk {
  int n, sub, t, tiles, length, subs;
  int held, held_from;

  __device__ __forceinline__ void hold(const AttentionParams& p, const Bars& bar, int lane) {
    held_from = n;
    held = n + lane < p.N ? length_at(p, bar, n + lane) : 0;
  }
  __device__ __forceinline__ void enter(const AttentionParams& p, const Bars& bar, int lane) {  // lengths of n, which has keys
    if (n >= p.N) {
      length = p.prefix;
      subs = p.H_k * p.prefix_blocks;
    } else {
      if (n - held_from >= 32) hold(p, bar, lane);
      length = __shfl_sync(0xffffffffu, held, n - held_from);
      subs = p.H_k * p.block_groups;
    }
    tiles = tiles_of(length);
  }
  __device__ __forceinline__ void next(const AttentionParams& p, const Bars& bar, int lane) {
    if (++t < tiles) return;
    t = 0;
    if (++sub < subs) return;
    sub = 0;
    ++n;
    while (n < p.N) {  // to the next sequence with keys
      if (n - held_from >= 32) hold(p, bar, lane);
      const unsigned some = __ballot_sync(0xffffffffu, held > 0) >> (n - held_from);
      if (some) {
        n += __ffs(some) - 1;
        break;
      }
      n = held_from + 32;
    }
    if (n > p.N) n = p.N;
    enter(p, bar, lane);
  }
};

// An 8 x 8 matrix of 16-bit elements, a lane's pair (t / 4, 2 (t % 4) + {0, 1}) turned into (2 (t % 4) + {0, 1}, t / 4).
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two weights as two pairs of the values' type whose sums they are, to 2^-15 (bf16) or 2^-21 (f16) of each: rounded once, they lose up to
// 2^-8 or 2^-11, as much as the output's own rounding.  A first part lies below its weight, so that the second is above zero, and an infinite
// value that meets both stays what it is.
template <bool F16>
__device__ __forceinline__ void split2(float a, float b, uint32_t& first, uint32_t& second) {
  const uint32_t below_a = max(__float_as_uint(a), 1u) - 1u, below_b = max(__float_as_uint(b), 1u) - 1u;   // (0 stays 0)
  if constexpr (F16) {
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(first) : "f"(__uint_as_float(below_b)), "f"(__uint_as_float(below_a)));
    const float2 x = unpack16<true>(first);
    second = pack16x2<true>(fmaxf(a - x.x, fminf(a, 0x1p-24f)), fmaxf(b - x.y, fminf(b, 0x1p-24f)));   // f16's smallest
  } else {
    first = __byte_perm(below_a, below_b, 0x7632);   // the upper halves
    second = pack16x2<false>(a - __uint_as_float(below_a & 0xffff0000u), b - __uint_as_float(below_b & 0xffff0000u));
  }
}

// 16 bytes to shared memory, zeros where there is nothing to copy.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(some ? 16 : 0) : "memory");
}
// Arrives (as one of those that the barrier counts) once this thread's copies so far are there.
__device__ __forceinline__ void arrive_copied(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The rows of a unit, for the worker of its group's block `side` (none behind the last block).
struct Unit {
  int tok0, head0, r0, rows, index;
  __device__ __forceinline__ Unit(const AttentionParams& p, const Walk& w, int side) {
    const bool own = w.n < p.N;
    const int head = own ? over(w.sub, p.by_groups) : w.sub, block = (own ? (w.sub - head * p.block_groups) * p.blocks_aside : 0) + side;
    head0 = head * p.group;
    r0 = block * kRows;
    tok0 = own ? w.n * p.tokens : 0;
    rows = w.length > 0 ? min(kRows, (own ? p.tokens : p.N * p.tokens) * p.group - r0) : 0;
    index = own ? (w.n * p.H_k + head) * p.blocks + block : p.N * p.H_k * p.blocks + head;
  }
};

// The copying warp.
template <int kEights>
__device__ __forceinline__ void copy_tiles(const AttentionParams& p, uint8_t* smem, Bars& bar, Walk walk, int count, int side) {
  const int lane = threadIdx.x & 31, boxes = kTile / p.box_rows;
  const auto key_of = [&](const Walk& w) { return lane < boxes ? w.t * kTile + lane * p.box_rows : INT32_MAX; };  // the lane's box' first
  const auto page_of = [&](const Walk& w) -> int64_t {  // looked at only when its turn comes: it is on its way until then
    const int key = key_of(w);
    if (key >= w.length) return 0;
    const int at = over(key, p.by_page);
    return w.n < p.N ? index_at(p.table, p.table_dtype, w.n * p.table_st + at) : index_at(p.prefix_pages, p.prefix_dtype, at);
  };
  // What one worker alone reads is not seen again, and leaves its place in L2 to a prefix that others read many times: 256 sequences behind
  // 32768 shared keys read 428 MB of HBM, 640 without (335 is the least).
  const uint64_t policy = p.blocks_aside > 1 ? l2_evict_normal() : l2_evict_first();
  int64_t page = page_of(walk);
  int issued = 0;
  for (int k = 0; k < count; ++k) {
    const int stage = k % kStages;
    Walk ahead = walk;
    int64_t page_ahead = 0;
    if (k + 1 < count) {
      ahead.next(p, bar, lane);
      page_ahead = page_of(ahead);
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&bar.empty[stage], (k / kStages + 1) & 1, p.wait_ns))) {
      if (lane == 0) atomicOr(p.dev_err, kDevErrTimeout);
      break;
    }
    ++issued;
    const int key = key_of(walk);
    const bool has = key < walk.length, good = has && page >= 0 && page < p.pages, held = p.hold_copies && k == 0;
    const bool bad = __any_sync(0xffffffffu, has && !good);
    const unsigned some = __ballot_sync(0xffffffffu, good);
    uint8_t* tile = smem + stage * kTileBytes;
    uint64_t* full = &bar.full[stage];
    if (lane == 0) {
      bar.bad[stage] = bad;
      if (bad) atomicOr(p.dev_err, kDevErrPage);
      mbar_arrive_expect_tx(full, __popc(some) * p.box_rows * 512);
    }
    __syncwarp();
    if (good && !held) {
      const int row = key - over(key, p.by_page) * p.page_size, head = walk.n < p.N ? over(walk.sub, p.by_groups) : walk.sub;
      uint8_t* at = tile + lane * p.box_rows * 256;
      tma_load_5d(at, &p.tm_k, full, 0, row, 0, head, (int)page, policy);
      tma_load_5d(at + kKeysBytes, &p.tm_v, full, 0, row, 0, head, (int)page, policy);
    }
    if (k == 0 || walk.t == 0) {  // the queries: half a warp a row, whose place a lane of each half finds for all
      const Unit u(p, walk, side);
      const uint32_t to = smem_u32(smem + kStages * kTileBytes + stage * kQueryBytes);
      const int chunk = lane & 15, r = u.r0 + chunk, token = over(r, p.by_group);
      const int64_t place = chunk < u.rows ? (int64_t)(u.tok0 + token) * p.q_st + (int64_t)(u.head0 + r - token * p.group) * p.q_sh : 0;
#pragma unroll
      for (int j = 0; j < 4 * kEights; ++j) {
        const int i = 2 * j + (lane >> 4);
        const uint16_t* from = reinterpret_cast<const uint16_t*>(p.q) + __shfl_sync(0xffffffffu, place, i) + 8 * chunk;
        copy16(to + i * 256 + ((chunk ^ (i & 7)) << 4), from, i < u.rows);
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
    if (!(p.hold_copies && k == 0)) mbar_wait(&bar.full[k % kStages], (k / kStages) & 1, kAttentionWaitNs);
}

// What a unit costs a worker beside its tiles (its queries, its end), in tiles: shares that count it come out even for short sequences, too.
constexpr int kUnitCost = 2;
__device__ __forceinline__ uint32_t cost_of(int length) { return length > 0 ? tiles_of(length) + kUnitCost : 0; }

// Keeps the first lengths in `bar`.  Tiles and cost of all sequences, in the units of one (key head, row block), counted by the first 128 of kThreads threads that
// meet at barrier `id`; `before`: those of the sequences in front of the thread's own, which are `each` in a row.
struct Count {
  struct Sums { uint32_t tiles, cost; };
  Sums all = {0, 0}, before = {0, 0}, mine = {0, 0};
  int each = 0;
  __device__ __forceinline__ void make(const AttentionParams& p, Bars& bar, uint32_t* room, int tid, int id) {
    constexpr int kCounting = 32 * kWarps;
    each = (p.N + kCounting - 1) / kCounting;
    if (tid < kCounting)
      for (int i = 0, n = tid * each; i < each && n < p.N; ++i, ++n) {
        const int length = length_of(p, n);
        if (n < kHeld) bar.lengths[n] = length;
        mine.tiles += tiles_of(length);
        mine.cost += cost_of(length);
      }
    Sums upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto.tiles, d), y = __shfl_up_sync(0xffffffffu, upto.cost, d);
      if ((tid & 31) >= d) { upto.tiles += x; upto.cost += y; }
    }
    Sums* sums = reinterpret_cast<Sums*>(room);
    if (tid < kCounting && (tid & 31) == 31) sums[tid >> 5] = upto;
    named_sync(id, kThreads);
    before = {upto.tiles - mine.tiles, upto.cost - mine.cost};
    for (int w = 0; w < kWarps; ++w) {
      if (w < tid >> 5) { before.tiles += sums[w].tiles; before.cost += sums[w].cost; }
      all.tiles += sums[w].tiles;
      all.cost += sums[w].cost;
    }
    fence_proxy_async_smem();   // tensor copies come over the room, behind the next barrier
  }
};
// The cost of everything that workers of the own pages walk, the prefix of few rows behind the sequences.
__device__ __forceinline__ uint32_t whole_cost(const AttentionParams& p, const Count& counted) {
  return counted.all.cost * p.H_k * p.block_groups + (p.prefix ? cost_of(p.prefix) * p.H_k * p.prefix_blocks : 0);
}

// Of the cost's point `at` in a sequence whose units begin at `from`, each of `tiles` tiles, after `index` tiles.
__device__ __forceinline__ Place place_in(uint32_t n, uint32_t at, uint32_t tiles, uint32_t index) {
  const uint32_t cost = tiles + kUnitCost, sub = at / cost, in = at - sub * cost, t = in > kUnitCost ? in - kUnitCost : 0;
  return {n, sub, t, index + sub * tiles + t};
}

// A worker for units of up to 8 kEights rows: `tid` below kThreads, the tiles counted by just these threads, ring and barriers of its own
// (initialised here), its number (blocks_aside in a row have the same share), how many shares there are.  `id`: a
// barrier of its own.  kBeside: a prefix on the tensor cores adds to the same outputs.
template <bool F16, int kEights, bool kBeside>
__device__ __forceinline__ void run_worker(const AttentionParams& p, uint8_t* smem, int tid, const Count& counted, int worker, int share_count, int id) {
  Bars& bar = bars_of(smem);
  const int lane = tid & 31, warp = tid >> 5, subs = p.H_k * p.block_groups;
  const int share = worker / p.blocks_aside, side = worker - share * p.blocks_aside;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.full[i], 33);     // the copying warp's lanes, and one of them for the tensor copies
      mbar_init(&bar.empty[i], kWarps);
    }
    mbar_init(&bar.joined, kWarps);
    fence_mbar_init();
  }
  // The share's two ends are looked up by the threads that counted the sequences where they lie.  (An end of everything lies nowhere: all
  // tiles are before it.)
  const Shares shares(whole_cost(p, counted), share_count);
  const uint32_t prefix_tiles = tiles_of(p.prefix), own_cost = counted.all.cost * subs, own_tiles = counted.all.tiles * subs;
#pragma unroll
  for (int end = 0; end < 2; ++end) {
    const uint32_t at = shares.from(share + end);
    if (tid < 32 * kWarps && counted.before.cost * subs <= at && at < (counted.before.cost + counted.mine.cost) * subs) {
      uint32_t cost = counted.before.cost * subs;
      Place place = {(uint32_t)p.N, 0, 0, counted.before.tiles * subs};
      for (int n = tid * counted.each; n < p.N; ++n) {
        const int length = length_at(p, bar, n);
        const uint32_t next = cost + cost_of(length) * subs;
        if (at < next) {
          place = place_in(n, at - cost, tiles_of(length), place.index);
          break;
        }
        cost = next;
        place.index += tiles_of(length) * subs;
      }
      bar.found[end] = place;
    }
    if (tid == 0 && at >= own_cost) {
      if (prefix_tiles && p.prefix_blocks && at < own_cost + (prefix_tiles + kUnitCost) * p.H_k * p.prefix_blocks) bar.found[end] = place_in(p.N, at - own_cost, prefix_tiles, own_tiles);
      else bar.found[end] = {0, 0, 0, own_tiles + (p.prefix_blocks ? prefix_tiles * p.H_k * p.prefix_blocks : 0)};
    }
  }
  named_sync(id, kThreads);
  const int count = (int)(bar.found[1].index - bar.found[0].index);
  if (count <= 0) return;   // a share that is nothing but a unit's cost
  Walk take;
  take.n = (int)bar.found[0].n;
  take.sub = (int)bar.found[0].sub;
  take.t = (int)bar.found[0].t;
  take.hold(p, bar, lane);
  take.enter(p, bar, lane);
  if (warp == kWarps) {
    copy_tiles<kEights>(p, smem, bar, take, count, side);
    return;
  }

  // All four warps walk the same units whatever happens on the way, so that they meet at the same ends.  (Lengths that someone changes
  // meanwhile could part them; the wait at an end has its limit, too.)
  const int mi = lane >> 3, mj = lane & 7;
  // a warp's 16 rows in a tile of boxes: where they begin, how far the second eight and the second half of a row are
  const auto rows_of = [](int w, int box) { return (w * kWarpKeys & -box) * 256 + (w * kWarpKeys & (box - 1)) * 128; };
  const auto eights_of = [](int box) { return box > 8 ? 1024 : 2048; };
  bool dead = false;
  int k = 0, stage = 0;
  uint32_t phase = 0, piece = 0;
  while (k < count) {  // the share's piece of a unit
    const bool own = take.n < p.N, starts = take.t == 0;
    const int tiles = max(1, min(take.tiles - take.t, count - k));   // lengths that change meanwhile do not keep it here
    bool unit_bad = false;
    uint32_t q[kEights][8][2];
    float base[kEights][2], sum[kEights][2], o[kEights][8][4] = {};   // rows 8 g + 2 (t % 4) + {0, 1}; o: values 16 j + t / 4 (+ 8)
#pragma unroll
    for (int g = 0; g < kEights; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e) { base[g][e] = -INFINITY; sum[g][e] = 0.f; }
#pragma unroll 1
    for (int i = 0;; ++i) {
      const uint32_t tile = smem_u32(smem) + stage * kTileBytes;
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(&bar.full[stage], phase, p.wait_ns))) {
        dead = true;
        if (lane == 0) atomicOr(p.dev_err, kDevErrTimeout);
      }
      if (i == 0) {
        const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int g = 0; g < kEights; ++g) {
          const uint32_t at = smem_u32(smem) + kStages * kTileBytes + stage * kQueryBytes + (8 * g + mj) * 256;
#pragma unroll
          for (int kk = 0; kk < 8; kk += 2) {
            uint32_t x[4];
            ldmatrix_x4(at + (((2 * kk + mi) ^ mj) << 4), x);
            q[g][kk][0] = x[0] ^ flip;
            q[g][kk][1] = x[1] ^ flip;
            q[g][kk + 1][0] = x[2] ^ flip;
            q[g][kk + 1][1] = x[3] ^ flip;
          }
        }
      }
      unit_bad |= dead || bar.bad[stage];
      const int key0 = take.t * kTile + warp * kWarpKeys, valid = min(kWarpKeys, take.length - key0);
      if (valid > 0 && !unit_bad) {
        const int box = here(p.box_rows), eights = eights_of(box), halves = box * 128;
        const uint32_t kb = tile + rows_of(warp, box), vb = kb + kKeysBytes;
        // Fragments are loaded ahead of the products that take them, the first of the values' before the weights are made.
        // (A row's chunk c of 16 bytes lies at c ^ row % 8: only these bits of an address change from step to step.)
        const uint32_t keys_at = kb + (mi & 1) * eights + mj * 128 + (((mi >> 1) ^ mj) << 4), values_at = vb + (mi >> 1) * eights + mj * 128 + (((mi & 1) ^ mj) << 4);
        const auto load_keys = [&](int kk, uint32_t (&to)[4]) { ldmatrix_x4((keys_at ^ ((kk & 3) << 5)) + (kk >> 2) * halves, to); };
        const auto load_values = [&](int j, uint32_t (&to)[4]) { ldmatrix_x4_trans((values_at ^ ((j & 3) << 5)) + (j >> 2) * halves, to); };
        float acc[kEights][2][4] = {};  // even and odd steps; (key t / 4, both rows), (key t / 4 + 8, both rows)
        constexpr int kAhead = kEights == 1 ? 2 : 1;   // as registers allow
        uint32_t f[kAhead + 1][4];
#pragma unroll
        for (int kk = 0; kk < kAhead; ++kk) load_keys(kk, f[kk]);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          if (kk + kAhead < 8) load_keys(kk + kAhead, f[(kk + kAhead) % (kAhead + 1)]);
#pragma unroll
          for (int g = 0; g < kEights; ++g) mma16<F16>(acc[g][kk & 1], f[kk % (kAhead + 1)], q[g][kk][0], q[g][kk][1]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) load_values(j, f[j]);
        float w[kEights][4];
        const int tail = own && p.tokens > 1 ? max(0, take.length - p.tokens + 1) : take.length;  // keys from here on are not for all rows
#pragma unroll
        for (int g = 0; g < kEights; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) w[g][e] = (acc[g][0][e] + acc[g][1][e]) * (fabsf(p.scale) * kLog2e);
        if (key0 + kWarpKeys > tail) {
          const Unit u(p, take, side);
          const int at_lane = here(lane);
#pragma unroll
          for (int g = 0; g < kEights; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + at_lane / 4 + 8 * (e >> 1), r = u.r0 + 8 * g + 2 * (at_lane & 3) + (e & 1);
              const int seen = own ? take.length - p.tokens + 1 + over(r, p.by_group) : take.length;
              if (key >= min(seen, take.length)) w[g][e] = -INFINITY;
            }
        }
        bool moves = false;
#pragma unroll
        for (int g = 0; g < kEights; ++g)
#pragma unroll
          for (int e = 0; e < 2; ++e) moves |= fmaxf(w[g][e], w[g][e + 2]) > base[g][e] + (kRoom + kBias<F16>);
        if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
          for (int g = 0; g < kEights; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(w[g][e], w[g][e + 2]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              const float now = fmaxf(base[g][e], top - kBias<F16>);
              const float keep = now == -INFINITY || now == base[g][e] ? 1.f : exp2_fast(base[g][e] - now);
              base[g][e] = now;
              sum[g][e] *= keep;
              if (i == 0) continue;   // all zeros
#pragma unroll
              for (int j = 0; j < 8; ++j) { o[g][j][e] *= keep; o[g][j][e + 2] *= keep; }
            }
        }
#pragma unroll
        for (int g = 0; g < kEights; ++g)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float from_base = base[g][e] == -INFINITY ? 0.f : base[g][e];
            w[g][e] = exp2_fast(w[g][e] - from_base);
            w[g][e + 2] = exp2_fast(w[g][e + 2] - from_base);
            sum[g][e] += w[g][e] + w[g][e + 2];
          }
        // What must not be seen must not meet the products, be its weight zero: an infinity would leave a NaN.  Places behind the
        // last key are cleared.  Keys that only some rows see seldom hold anything but numbers; where they do, they are
        // added by hand and cleared, too.
        int clean = valid;
        if (key0 + kWarpKeys > tail) {
          const int some = min(valid, max(0, tail - key0));  // keys that all rows see
          bool odd = false;
          for (int n = lane; n < (valid - some) * 16; n += 32) {
            const int j = some + n / 16, chunk = n % 16;
            uint32_t x[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(vb + (chunk >> 3) * halves + (j >> 3) * eights + (j & 7) * 128 + ((chunk & 7) << 4)));
            constexpr uint32_t kTop = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll
            for (int e = 0; e < 4; ++e) odd |= (x[e] & kTop) == kTop || (x[e] >> 16 & kTop) == kTop;
          }
          if (__any_sync(0xffffffffu, odd)) clean = some;
        }
        if (clean < kWarpKeys) {
          const Unit u(p, take, side);
          const int at_lane = here(lane);
#pragma unroll 1
          for (int j = clean; j < valid; ++j) {
            const int from = ((j & 7) << 2) | (at_lane & 3);
#pragma unroll
            for (int g = 0; g < kEights; ++g)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float pj = __shfl_sync(0xffffffffu, j < 8 ? w[g][e] : w[g][e + 2], from);
                const int r = u.r0 + 8 * g + 2 * (at_lane & 3) + e;
                if (key0 + j >= take.length - p.tokens + 1 + over(r, p.by_group)) continue;  // not seen
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                  const int value = 8 * n + at_lane / 4;
                  uint16_t x;
                  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(vb + (n >> 3) * halves + (j >> 3) * eights + (j & 7) * 128 + (((n & 7) ^ (j & 7)) << 4) + 2 * (value & 7)));
                  float& to = o[g][n >> 1][e + 2 * (n & 1)];
                  to = fmaf(pj, unpack16<F16>((uint32_t)x).x, to);
                }
              }
          }
          __syncwarp();
          for (int n = lane; n < (kWarpKeys - clean) * 16; n += 32) {
            const int j = clean + n / 16, chunk = n % 16;
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (chunk >> 3) * halves + (j >> 3) * eights + (j & 7) * 128 + ((chunk & 7) << 4)), "r"(0) : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
#pragma unroll
          for (int g = 0; g < kEights; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (at_lane / 4 + 8 * (e >> 1) >= clean) w[g][e] = 0.f;
#pragma unroll
          for (int j = 0; j < kAhead; ++j) load_values(j, f[j]);
        }
        // Weights go into the sums as two parts (split2) where one block of rows reads the keys: HBM bounds that, and it costs
        // little (256 sequences of 8192 keys and 8 rows 638 us with and without, 128 of 4096 keys and 16 rows 173 us instead of 172, one tile 8.4
        // instead of 8.3).  Where several blocks read them, the products bound the kernel, and weights are rounded once: 64 sequences of 1500 keys and 64
        // rows take 84 us instead of 97, and outputs are 1.35 times as far off as with a rounding of the output alone.  So they are beside a
        // prefix on the tensor cores, whose weights are rounded once, too (48 sequences of 16 rows and 2000 keys behind 16384: 50 us instead of 54).
        const auto add = [&](auto of) {
          constexpr int kParts = decltype(of)::value;
          uint32_t b[kEights][2][2];
#pragma unroll
          for (int g = 0; g < kEights; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t part[2];
              if constexpr (kParts == 2) split2<F16>(w[g][2 * e], w[g][2 * e + 1], part[0], part[1]);
              else part[0] = pack16x2<F16>(w[g][2 * e], w[g][2 * e + 1]);
#pragma unroll
              for (int n = 0; n < kParts; ++n) b[g][n][e] = transposed(part[n]);
            }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j + kAhead < 8) load_values(j + kAhead, f[(j + kAhead) % (kAhead + 1)]);
#pragma unroll
            for (int g = 0; g < kEights; ++g)
#pragma unroll
              for (int n = 0; n < kParts; ++n) mma16<F16>(o[g][j], f[j % (kAhead + 1)], b[g][n][0], b[g][n][1]);
          }
        };
        if (!kBeside && (kEights == 1 || p.blocks == 1)) add(std::integral_constant<int, 2>{});
        else add(std::integral_constant<int, 1>{});
      }
      if (i + 1 == tiles) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.empty[stage]);
      ++take.t;
      if (++stage == kStages) { stage = 0; phase ^= 1; }
    }
    // The warps' parts of the piece come together over its last tile: a row of sums takes half of one of the eight kilobytes that the warp's
    // keys and values were in, the columns by eights turned by the row.
    const bool ends = take.t + 1 == take.tiles, whole = starts && ends;
    const int at_lane = here(lane), at_tid = here(tid);
    float2(&ml)[kWarps][kRows] = bar.ml[piece & 1];
    uint8_t* const tile = smem + stage * kTileBytes;
    const int box = here(p.box_rows), eights = eights_of(box), halves = box * 128;
#pragma unroll
    for (int g = 0; g < kEights; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum[g][e] += __shfl_xor_sync(0xffffffffu, sum[g][e], d);
        if (at_lane < 4) ml[warp][8 * g + 2 * at_lane + e] = make_float2(base[g][e], unit_bad ? kAttentionBad : sum[g][e]);
      }
    __syncwarp();
    float* const to = reinterpret_cast<float*>(tile + rows_of(warp, box) + (at_lane >> 1 & 1) * halves + (at_lane & 1) * eights) + at_lane / 4;
#pragma unroll
    for (int g = 0; g < kEights; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int n = 0; n < 16; ++n)
          to[g * (kKeysBytes / 4) + e * kHeadDim + (n ^ (at_lane & 3)) * 8] = o[g][n >> 1][e + 2 * (n & 1)];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.joined);
    if (!dead && !__all_sync(0xffffffffu, mbar_wait(&bar.joined, piece & 1, p.wait_ns))) {
      dead = true;
      if (lane == 0) atomicOr(p.dev_err, kDevErrTimeout);
    }
    ++piece;
    const Unit u(p, take, side);
    if (tid == 0 && u.rows > 0) {
      if (starts) p.first_worker[u.index] = worker;
      if (ends) p.last_worker[u.index] = worker;
    }
    const int64_t slot = whole ? 2 * p.workers + (int64_t)u.index : 2 * worker + (starts ? 1 : 0);
    const int cg = at_tid & 15, row0 = at_tid / 16;
    const bool turned = cg & 4;  // these take their second four columns first, so that eight lanes meet in no bank
    const float* const from = reinterpret_cast<const float*>(tile + (row0 >> 2 & 1) * halves + (row0 >> 1 & 1) * eights + (row0 & 1) * 512) + (cg ^ (row0 >> 1 & 3)) * 8;
    float x[kEights][8], top[kEights], l[kEights];
    bool bad = dead;
#pragma unroll
    for (int g = 0; g < kEights; ++g) {
      const int row = row0 + 8 * g;
      float2 of[kWarps];
      top[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        of[w] = ml[w][row];
        top[g] = fmaxf(top[g], of[w].x);
        bad |= of[w].y == kAttentionBad;
      }
      const float from_base = top[g] == -INFINITY ? 0.f : top[g];
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_fast(of[w].x - from_base);
        const float4* y = reinterpret_cast<const float4*>(from + (g * kKeysBytes + rows_of(w, box)) / 4);
        const float4 y0 = y[turned], y1 = y[!turned];
        l[g] = fmaf(f, of[w].y, l[g]);
        a = make_float4(fmaf(f, y0.x, a.x), fmaf(f, y0.y, a.y), fmaf(f, y0.z, a.z), fmaf(f, y0.w, a.w));
        b = make_float4(fmaf(f, y1.x, b.x), fmaf(f, y1.y, b.y), fmaf(f, y1.z, b.z), fmaf(f, y1.w, b.w));
      }
      x[g][0] = turned ? b.x : a.x; x[g][1] = turned ? b.y : a.y; x[g][2] = turned ? b.z : a.z; x[g][3] = turned ? b.w : a.w;
      x[g][4] = turned ? a.x : b.x; x[g][5] = turned ? a.y : b.y; x[g][6] = turned ? a.z : b.z; x[g][7] = turned ? a.w : b.w;
    }
    // the tile is given back, and the warps go on, before what they have is on its way to memory
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.empty[stage]);
#pragma unroll
    for (int g = 0; g < kEights; ++g) {
      const int row = row0 + 8 * g, r = u.r0 + row;
      const bool some = row < u.rows;
      if (whole && !p.prefix) {
        const bool none = top[g] == -INFINITY && l[g] == 0.f;
        const float inv = none ? 0.f : inverse(l[g]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[g][e] *= inv;
        const int of_unit = over(r, p.by_group), head = u.head0 + r - of_unit * p.group;
        const int64_t token = u.tok0 + of_unit;
        const uint4 y = pack16x8<F16>(x[g]);
        if (some && !bad) *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + token * p.o_st + head * p.o_sh + 8 * cg) = y;
        if (some && !bad && p.lse && cg == 0)
          p.lse[token * p.lse_st + head] = none ? -INFINITY : ((top[g] == -INFINITY ? 0.f : top[g]) + log2f(l[g])) * kLn2;
      } else if (some) {
        float4* y = reinterpret_cast<float4*>(p.part_o + (slot * p.block_rows + row) * kHeadDim + 8 * cg);
        y[0] = make_float4(x[g][0], x[g][1], x[g][2], x[g][3]);
        y[1] = make_float4(x[g][4], x[g][5], x[g][6], x[g][7]);
        if (cg == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * p.block_rows + row) * 2) = make_float2(top[g], bad ? kAttentionBad : l[g]);
      }
    }
    k += tiles;
    if (++stage == kStages) { stage = 0; phase ^= 1; }
    if (k < count) take.next(p, bar, lane);
  }
}

}  // namespace own
}  // namespace gdn
