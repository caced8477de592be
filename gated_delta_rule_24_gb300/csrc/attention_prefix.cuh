// Softmax attention of many rows over the prefix that they share, for sm_103a: the part of the paged
// attention (attention.cu) that reads keys and values once for the whole batch, as one CTA does its share of it.
//
//   s_j = scale q . k_j,   (base, sum_j 2^(s_j log2(e) - base), sum_j 2^(s_j log2(e) - base) v_j)
//
// All rows of a key head (sequences x tokens x its query heads) see all keys, so there is nothing to mask but what lies
// behind the prefix in its last tile.  Every key costs 4 x 128 flops a row against 512 bytes: from some
// 300 rows on the tensor cores bound it.  A CTA takes 256 rows as two tiles of 128, A and B, against
// 128 keys at a time:
//
//   S = Q K^T (tcgen05, both operands in shared memory, S in TMEM),
//   P = 2^(S - base) by one thread a row, 16-bit, to TMEM in S's place,
//   O += P V (tcgen05, P from TMEM, O in TMEM),
//
// and while four warps make A's weights, the tensor cores are at B's products, and the other way round.
// (P comes in two halves, and the first goes into the product while the second is made.)  A
// base moves only when a score exceeds the largest before it by 2^8, so that O is seldom read back to be scaled: the weights
// grow to 2^8 at most (2^14 in f16, attention_common.cuh), which changes no rounding.  When S of a tile is there, all products issued before it
// are done, so a row's thread may scale O then without a hand-off of its own.
//
// P is rounded once to the values' type, as the product wants both operands of one type; the sum of weights is of what they were before, in
// f32.  That costs outputs up to u sum w |v| (2.2e-3 of the output instead of 1.65e-3 in bf16, its own rounding included).  A second
// product with the rest would take the tensor cores 1030 clocks more for each 128 keys of 256 rows, beside the 2048 of the others.
//
// Where a unit has no more than 128 rows, A and B are the same rows and take every other tile of keys, and their sums come
// together at the end of a piece.
//
// Units are (key head, 256 rows), a unit's tiles of 128 keys come one behind the other, and all units'
// tiles are cut into equal shares for the SMs; the parts are joined by attention.cu's second kernel.
//
// Measured: 128 keys of 256 rows take an SM 2700 to 2870 clocks (1.4 us) of the 2048 that the products alone need: a row's weights take 1570
// from its scores, and the products of a tile 1310 then, 1030 where nothing else uses TMEM and shared memory.  256 sequences of 8 rows over 32768 shared keys on 4 key heads,
// each with some own pages: 123 us in all in a graph, up to 133 as a call among others.
#pragma once
#include <type_traits>

#include "attention_common.cuh"

namespace gdn {
namespace prefix {

constexpr int kThreads = 384;                 // two groups of four warps for the weights, one with the copies and the products
constexpr int kHalf = 16384;                  // 128 rows of 64 values
constexpr int kTileBytes = 2 * kHalf;
constexpr int kStages = 2;                    // of keys, and of values
constexpr int kQ = 0, kK = 2 * kTileBytes, kV = kK + kStages * kTileBytes, kBars = kV + kStages * kTileBytes;
constexpr int kBytes = kBars + 4096;

constexpr uint32_t kS = 0, kO = 256;          // TMEM columns: S of A and B (and P over it), O of A and B
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n.reg .b64 x, y;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Waits for this thread's loads from TMEM, and keeps what uses these registers behind the wait.
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

struct Bars {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], done;
  uint32_t tmem, bad;
  float2 ml[2][128];   // base and sum of A's and B's rows where they are the same
};

static_assert(sizeof(Bars) <= kBytes - kBars, "room for them");

// A unit's tiles, and what it costs a worker beside them (rows of Q in, sums out: some 6 us against 1.4 us for a tile).
constexpr uint32_t kUnitCost = 4;
struct Steps {
  uint32_t tiles, cost;   // of a unit
  Shares shares;
  __device__ __forceinline__ Steps(const AttentionParams& p, int workers)
      : tiles((p.prefix + kPrefixKeys - 1) / kPrefixKeys), cost(tiles + kUnitCost), shares(p.H_k * p.prefix_units * cost, workers) {}
};

// The share of a worker, and the pieces of units that it makes.
struct Share {
  uint32_t at, end, tiles, cost;
  __device__ __forceinline__ Share(const Steps& s, int worker) : at(s.shares.from(worker)), end(s.shares.from(worker + 1)), tiles(s.tiles), cost(s.cost) {}
  int unit, t0, n;  // the piece: tiles t0 .. t0 + n - 1 of the unit
  __device__ __forceinline__ bool next() {
    while (at < end) {
      const uint32_t u = at / cost, to = min(end, (u + 1) * cost), a = at - u * cost, b = to - u * cost;
      unit = (int)u;
      t0 = a > kUnitCost ? a - kUnitCost : 0;
      n = (b > kUnitCost ? b - kUnitCost : 0) - t0;
      at = to;
      if (n > 0) return true;
    }
    return false;
  }
};

template <bool F16>
__device__ __forceinline__ void run_worker(const AttentionParams& p, uint8_t* smem, int worker, int workers) {
  Bars& bar = *reinterpret_cast<Bars*>(smem + kBars);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = warp >> 2;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 128);
      mbar_init(&bar.s_full[i], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&bar.p_full[i][h], 128);
      mbar_init(&bar.o_full[i], 1);
    }
    mbar_init(&bar.done, 1);
    fence_mbar_init();
    bar.bad = 0;
  }
  if (warp == 9) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  const uint64_t limit = p.wait_ns;
  const int rows_all = p.N * p.tokens * p.group;
  Share share(Steps(p, workers), worker);
  const auto turns = [&] { return rows_all - (share.unit - over(share.unit, p.by_units) * p.prefix_units) * kPrefixRows <= 128; };  // A and B take turns at the tiles

  if (group == 2) {
    if (warp == 8) {  // copies
      const int box = p.prefix_box, boxes = kPrefixKeys / box;
      bool dead = false;
      int step = 0, issued[2] = {0, 0};
      auto page_of = [&](int t) -> int64_t {
        const int key = t * kPrefixKeys + lane * box;
        if (lane >= boxes || key >= p.prefix) return -2;
        const int64_t page = index_at(p.prefix_pages, p.prefix_dtype, over(key, p.by_page));
        return page < 0 || page >= p.pages ? -1 : page;
      };
      while (!dead && share.next()) {
        const int head = over(share.unit, p.by_units);
        int64_t page = page_of(share.t0);
        for (int i = 0; i < share.n && !dead; ++i, ++step) {
          const int t = share.t0 + i, st = step % kStages;
          const int64_t ahead = i + 1 < share.n ? page_of(t + 1) : -2;
          const unsigned some = __ballot_sync(0xffffffffu, page >= 0);
          if (__any_sync(0xffffffffu, page == -1) && lane == 0) {
            atomicOr(p.dev_err, kDevErrPage);
            atomicOr(&bar.bad, 1u);
          }
          const uint32_t bytes = __popc(some) * box * 256;
          const int key = t * kPrefixKeys + lane * box, row = key - over(key, p.by_page) * p.page_size;
          for (int kv = 0; kv < 2; ++kv) {
            uint64_t* full = kv ? &bar.v_full[st] : &bar.k_full[st];
            dead = dead || !__all_sync(0xffffffffu, mbar_wait(kv ? &bar.v_empty[st] : &bar.k_empty[st], (step / kStages + 1) & 1, limit));
            if (dead) break;
            if (lane == 0) mbar_arrive_expect_tx(full, bytes);
            __syncwarp();
            ++issued[kv];
            if (page >= 0 && !(p.hold_copies && step == 0)) {
              uint8_t* at = smem + (kv ? kV : kK) + st * kTileBytes + lane * box * 128;
              for (int half = 0; half < 2; ++half)
                tma_load_4d(at + half * kHalf, kv ? &p.tm_pv : &p.tm_pk, full, 64 * half, head, row, (int)page);
            }
            __syncwarp();
          }
          page = ahead;
        }
      }
      if (dead && lane == 0) atomicOr(p.dev_err, kDevErrTimeout);
      // every copy ends before the memory is another's
      for (int kv = 0; kv < 2; ++kv)
        for (int i = max(0, issued[kv] - kStages); i < issued[kv]; ++i)
          if (!(p.hold_copies && i == 0)) mbar_wait(kv ? &bar.v_full[i % kStages] : &bar.k_full[i % kStages], (i / kStages) & 1, kAttentionWaitNs);
    } else if (warp == 9) {  // products, by one thread from end to end: each elects, votes and branches of a warp would cost what a product does
      if (elect_one()) {
        bool dead = false;
        uint32_t step = 0, steps[2] = {0, 0}, pieces[2] = {0, 0};
        const uint32_t id_s = idesc_16_f32(F16, 128, 128, 0, 0, p.scale < 0.f);
        constexpr uint32_t id_o = idesc_16_f32(F16, 128, 128, 0, 1, 0);
        const uint64_t d_q = sdesc_sw128(smem_u32(smem + kQ), 16, 1024), d_k = sdesc_sw128(smem_u32(smem + kK), 16, 1024),
                       d_v = sdesc_sw128(smem_u32(smem + kV), kHalf, 1024);   // shared addresses count by 16 bytes in them
        using std::integral_constant;
        constexpr integral_constant<int, 0> kA{};
        constexpr integral_constant<int, 1> kB{};
        const auto wait = [&](uint64_t* b, uint32_t parity) {
          dead = dead || !mbar_wait(b, parity & 1, limit);
          tc_fence_after();
        };
        const auto commit = [&](uint64_t* b) {
          if (!dead) mma_commit(b);
        };
        const auto scores = [&](auto which, auto rows, uint32_t at) {  // S of A or B, with the rows of tile `rows`, of the keys of step `at`
          constexpr int x = decltype(which)::value, tile = decltype(rows)::value;
          const uint64_t a = d_q + tile * (kTileBytes >> 4), b = d_k + at % kStages * (kTileBytes >> 4);
          if (dead) return;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
            mma_ss(tmem + kS + 128 * x, a + off, b + off, id_s, kk > 0);
          }
          mma_commit(&bar.s_full[x]);
        };
        const auto values = [&](auto which, uint32_t at, bool more) {  // O of A or B, of the values of step `at`
          constexpr int x = decltype(which)::value;
          const uint32_t st = at % kStages;
          const uint64_t b = d_v + st * (kTileBytes >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wait(&bar.p_full[x][h], steps[x]);
            if (h == 0) wait(&bar.v_full[st], at / kStages);
            if (dead) return;
#pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              mma_ts(tmem + kO + 128 * x, tmem + kS + 128 * x + 8 * kk, b + kk * (2048 >> 4), id_o, kk > 0 || more);
          }
          ++steps[x];
        };
        while (!dead && share.next()) {
          const uint32_t n = share.n;
          if (turns()) {
            wait(&bar.q_full[0], pieces[0]++);
            const auto start = [&](auto which, uint32_t at) {
              wait(&bar.k_full[at % kStages], at / kStages);
              scores(which, kA, at);
              commit(&bar.k_empty[at % kStages]);
            };
            const auto tile = [&](auto which, uint32_t i) {
              const uint32_t at = step + i;
              values(which, at, i > 1);
              commit(&bar.v_empty[at % kStages]);
              if (i + 2 < n) start(which, at + 2);
              else commit(&bar.o_full[decltype(which)::value]);
            };
            start(kA, step);
            if (n > 1) start(kB, step + 1);
#pragma unroll 1
            for (uint32_t i = 0; i < n && !dead; i += 2) {
              tile(kA, i);
              if (i + 1 < n) tile(kB, i + 1);
            }
            step += n;
            continue;
          }
          wait(&bar.q_full[0], pieces[0]++);
          wait(&bar.k_full[step % kStages], step / kStages);
          scores(kA, kA, step);
          wait(&bar.q_full[1], pieces[1]++);
          scores(kB, kB, step);
          commit(&bar.k_empty[step % kStages]);
#pragma unroll 1
          for (uint32_t i = 0; i < n && !dead; ++i, ++step) {
            const uint32_t ahead = step + 1;
            const bool last = i + 1 == n;
            values(kA, step, i > 0);
            if (!last) {
              wait(&bar.k_full[ahead % kStages], ahead / kStages);
              scores(kA, kA, ahead);
            } else {
              commit(&bar.o_full[0]);
            }
            values(kB, step, i > 0);
            commit(&bar.v_empty[step % kStages]);
            if (!last) {
              scores(kB, kB, ahead);
              commit(&bar.k_empty[ahead % kStages]);
            } else {
              commit(&bar.o_full[1]);
            }
          }
        }
        if (dead) atomicOr(p.dev_err, kDevErrTimeout);
        // nothing is on its way to or from TMEM any more
        mma_commit(&bar.done);
        mbar_wait(&bar.done, 0, kAttentionWaitNs);
      }
      __syncwarp();
    }
  } else {
    const int x = group, i128 = tid & 127;  // tile A or B, the thread's row of it
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = tmem + kS + 128 * x + lanes, o_at = tmem + kO + 128 * x + lanes;
    const float c = fabsf(p.scale) * kLog2e;
    bool dead = false;
    uint32_t steps = 0, pieces = 0, first = 0;   // `first`: the piece's first step
    auto wait = [&](uint64_t* b, uint32_t parity) {
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(b, parity & 1, limit))) {
        dead = true;
        if (lane == 0) atomicOr(p.dev_err, kDevErrTimeout);
      }
    };
    for (; share.next(); first += share.n) {
      const bool turn = turns();
      const int unit_head = over(share.unit, p.by_units), unit_row = (share.unit - unit_head * p.prefix_units) * kPrefixRows, row0 = unit_row + (turn ? 0 : 128 * x), r = row0 + i128;
      if (!turn || x == 0) {  // the rows of Q, half a warp a row, all on their way at once
        const int head = unit_head * p.group, chunk = lane & 15;
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + 8 * chunk;
        const uint32_t to = smem_u32(smem + kQ + x * kTileBytes + (chunk >> 3) * kHalf);
#pragma unroll 4
        for (int j = 0; j < 16; ++j) {
          const int rr = (warp & 3) * 32 + 2 * j + (lane >> 4), row = row0 + rr, token = over(row, p.by_group);
          const bool some = row < rows_all;
          const uint16_t* from = some ? q + (int64_t)token * p.q_st + (int64_t)(head + row - token * p.group) * p.q_sh : q;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + sw128_chunk(rr, chunk & 7)), "l"(from), "r"(some ? 16 : 0) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(&bar.q_full[x]);
      }
      float base = -INFINITY;
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int i = turn ? x : 0; i < share.n; i += turn ? 2 : 1) {
        wait(&bar.s_full[x], steps++);
        if (dead) continue;
        tc_fence_after();
        // A row's scores pass twice, the second time as its weights are made: half of them stay in registers, P lies
        // over what was read, never over what is still to be.
        const int valid = p.prefix - (share.t0 + i) * kPrefixKeys;
        float top[4];
        uint32_t s0[32], s1[32], s2[32];
        auto largest = [&](int h, uint32_t (&s)[32]) {
          if (valid < kPrefixKeys) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * h + e >= valid) s[e] = 0xff800000u;
          }
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = __uint_as_float(s[e]);
#pragma unroll
          for (int e = 4; e < 32; ++e) y[e & 3] = fmaxf(y[e & 3], __uint_as_float(s[e]));
          top[h] = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        };
        tmem_ld32(s_at + 64, s0);
        tmem_ld32(s_at + 96, s1);
        loaded(s0);
        loaded(s1);
        largest(2, s0);
        largest(3, s1);
        tmem_ld32(s_at, s0);
        tmem_ld32(s_at + 32, s1);
        loaded(s0);
        loaded(s1);
        largest(0, s0);
        largest(1, s1);
        if (valid < kPrefixKeys && (x == 0 || turn)) {  // values of no key have a weight of zero, but must not be infinite either
          const uint32_t at = first + i;
          wait(&bar.v_full[at % kStages], at / kStages);
          uint8_t* v = smem + kV + (at % kStages) * kTileBytes;
          for (int e = i128; e < (kPrefixKeys - valid) * 16; e += 128)
            *reinterpret_cast<uint4*>(v + (e & 8 ? kHalf : 0) + (valid + e / 16) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          if (dead) continue;
        }
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
        if (__any_sync(0xffffffffu, high > base + (kRoom + kBias<F16>))) {
          const float now = fmaxf(base, high - kBias<F16>);
          const float keep = now == -INFINITY || now == base ? 1.f : exp2_fast(base - now);
          base = now;
          sum = mul2(sum, pair(keep));
          if (i > (turn ? 1 : 0)) {
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
              uint32_t o[32];
              tmem_ld32(o_at + 32 * h, o);
              loaded(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
              tmem_st32(o_at + 32 * h, o);
            }
          }
        }
        const float2 minus = pair(base == -INFINITY ? 0.f : -base), cc = pair(c);
        auto weights = [&](int h, uint32_t (&s)[32], bool masked) {
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * h + e >= valid) s[e] = 0xff800000u;
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 y = fma2(pair_at(&s[2 * e]), cc, minus);
            y.x = exp2_fast(y.x);
            y.y = exp2_fast(y.y);
            sum = add2(sum, y);
            w[e] = pack16x2<F16>(y);
          }
          tmem_st16(s_at + 16 * h, w);
        };
        tmem_ld32(s_at + 64, s2);
        weights(0, s0, false);
        loaded(s2);
        tmem_ld32(s_at + 96, s0);
        weights(1, s1, false);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_full[x][0]);
        weights(2, s2, valid < kPrefixKeys);
        loaded(s0);
        weights(3, s0, valid < kPrefixKeys);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_full[x][1]);
      }
      const bool some = !turn || x < share.n;  // tiles for this group
      if (some) wait(&bar.o_full[x], pieces++);
      tc_fence_after();
      const bool ends = share.t0 + share.n == (int)share.tiles, write = r < rows_all;
      if (tid == 0) {
        if (share.t0 == 0) p.prefix_first[share.unit] = worker;
        if (ends) p.prefix_last[share.unit] = worker;
      }
      const int64_t slot = share.t0 == 0 && ends ? 2 * (int64_t)p.prefix_workers + share.unit : 2 * (int64_t)worker + (share.t0 == 0 ? 1 : 0);
      const int row = turn ? i128 : 128 * x + i128;
      float* y = p.prefix_o + slot * kPrefixRows * kHeadDim + row * 8;   // by eights of columns: a warp writes 1 KB in a row
      const auto store = [&](int h, const uint32_t (&o)[32]) {
        if (!write) return;
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(y + (4 * h + e / 8) * kPrefixRows * 8),
                       "r"(o[e]), "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]), "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7])
                       : "memory");
      };
      float total = sum.x + sum.y;
      if (dead || *reinterpret_cast<volatile uint32_t*>(&bar.bad)) total = kAttentionBad;
      if (!turn) {
        if (!dead) {
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            uint32_t o[32];
            tmem_ld32(o_at + 32 * h, o);
            loaded(o);
            store(h, o);
          }
        }
      } else {  // the sums of A and B come together, half the columns in each group
        bar.ml[x][i128] = make_float2(base, total);
        tc_fence_before();
        named_sync(1, 256);
        tc_fence_after();
        const float2 other = bar.ml[x ^ 1][i128];
        const bool any_bad = total == kAttentionBad || other.y == kAttentionBad;
        const float now = fmaxf(base, other.x), from_base = now == -INFINITY ? 0.f : now;
        const float mine = exp2_fast(base - from_base), theirs = exp2_fast(other.x - from_base);
        if (!any_bad) {
          const uint32_t o_theirs = tmem + kO + 128 * (x ^ 1) + lanes;
          const bool have_mine = some, have_theirs = (x ^ 1) < share.n;   // O of a group without tiles holds anything
#pragma unroll 1
          for (int h = 2 * x; h < 2 * x + 2; ++h) {
            uint32_t o[32], o2[32];
            tmem_ld32(o_at + 32 * h, o);
            tmem_ld32(o_theirs + 32 * h, o2);
            loaded(o);
            loaded(o2);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint((have_mine ? mine * __uint_as_float(o[e]) : 0.f) + (have_theirs ? theirs * __uint_as_float(o2[e]) : 0.f));
            store(h, o);
          }
        }
        base = now;
        total = any_bad ? kAttentionBad : mine * total + theirs * other.y;
        tc_fence_before();
        named_sync(1, 256);   // before either O is another's
        tc_fence_after();
      }
      if (write && (!turn || x == 0)) *reinterpret_cast<float2*>(p.prefix_ml + 2 * (slot * kPrefixRows + row)) = make_float2(base, total);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

}  // namespace prefix
}  // namespace gdn
