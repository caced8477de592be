// Linear attention with a decay over packed sequences, sm_103a: for each sequence and head,
// with the state S (V-major 128 x 128: row = value index, column = key index),
//
//   S_t = g_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t.
//
// Chunk form, 128 tokens at a time (i, j tokens of the chunk, G = cumsum(log2 g)):
//
//   P_ij = scale 2^(G_i - G_j) (q_i . k_j)   for j <= i, else 0
//   O    = scale diag(2^G) Q S^T + P V
//   S   <- 2^(G_last) S + V_d^T K,           V_d = diag(2^(G_last - G)) V
//
// Four products of 128 x 128 x 128 on tcgen05 (the last one two or three times, see below) against
// 128 KB of q, k, v and o.  At 6.8 TB/s an SM of 152 gets its 128 KB in 2.9 us, and the products
// take 1.6 us (two terms; 592 cycles a product with its A operand in TMEM, 853 with A in shared memory,
// so that all four have A there): the bytes bound it where every SM is busy and heads share nothing,
// and otherwise the chain of roles that a chunk goes through does.
//
// A CTA an SM walks (sequence, head) units chunk by chunk.  Roles (24 warps; 80 registers a thread):
//   warp 0      unit records, TMA loads of Q, K, V (K and V in two stages) and of states;
//   warp 1      issues the products of a chunk: Q K^T, Q S^T, V_d^T K, P V.  P is built while Q S^T
//               and V_d^T K run; the state is read and V_d of the next chunk made while P V and the next
//               Q K^T run;
//   warp 2      the gates: prefix and suffix sums of log2 g, one chunk ahead;
//   warp 3      stores of output tiles (TMA, or rows where a sequence ends inside) and of states;
//   warps 4-11  two threads a token: Q from shared memory to TMEM, P (scores times decay, masked, back to
//               TMEM), Q S^T times scale 2^G_i in place, and the output tile;
//   warps 12-15 one thread a value row: before a chunk's V_d^T K adds to it, the state in TMEM goes times
//               the chunk's decay, and as a 16-bit copy to shared memory for Q S^T; f32 states stay in
//               these warps' registers, and take from TMEM what each chunk adds;
//   warps 16-23 V_d: transposed fragments of V times d, to TMEM.
// Hand-offs are mbarriers, every wait is bounded and ends early when any role gave up.  With all
// roles resident the instruction cache is short: loops are rolled up where that measured faster
// (P in rolled blocks of 16 columns: 16 x 4096 tokens on 32 heads 341 -> 322 us), and launches that
// meet no f32 state, or whose CTAs take no units over, are compiled without the code for that (1024
// short prompts 680 -> 640 us, 650 -> 638).
//
// TMEM is full: the scores (then P), the output, the state (128 columns each), Q and V_d (64
// each).  Further parts of V_d go where Q was, once Q S^T has read it, and between the blocks of P.
//
// Too few units for the SMs: sequences are cut into segments (decay_splits).  One launch makes the
// states that the segments add (K and V alone), the join chains them in f32, and the main
// launch runs all segments from those.
//
// Measured (bf16 unless stated; time of the launches in short bursts, share of 6.8 TB/s in the bytes that have to
// move; back to back for seconds the power limit adds 2 to 5 % to the first four):
//   12800 tokens, 152 heads, none shared:  294 us, 6.6 TB/s (98 %); 333 with f32 states
//   16 x 4096, 16 q/k and 32 v heads, bf16 states: 314 us (77 %): 512 units are 3.4 rounds of 152; f32 states 407
//   2 x 65536, 16 and 32 heads, f32 states: 1055 us (45 %); 7 segments, K and V read twice, three terms
//   32000 tokens, 8 heads, f16: 85 to 93 us (45 to 42 %); 31 us states, 7 join, the rest outputs
//   1024 prompts of 136 on average, 8 and 16 heads, bf16 states: 637 us (65 %); 1.6 chunks a unit; f32 states 857
//   one chunk of a unit alone: 2.2 us with two terms (f16 and f32 states 2.5), 2.8 with three
// Tensor pipe 54 % busy, issue slots 53 %, 60 % of DRAM (8 x 4096, 16 and 32 heads): a chunk takes
// 4300 cycles at 2960 of products, the rest is hand-offs of 300 to 450 cycles between roles.
//
// Precision: P and the copy of S are rounded to the 16-bit type of q, k, v (as the output is);
// everything else that is summed is f32 (by the tensor cores towards zero: see apart).  V_d would
// put its rounding straight into the state, so it enters as the sum of 16-bit terms, each the
// rounding of what is left: two (16 bits bf16, 22 bits f16, where v_scale keeps them in f16's
// range), or three for bf16 inputs whose state stays in f32, which then is as exact as f32 sums
// are.  The third term costs 0.5 us a chunk where SMs are not kept busy by bytes.
//
// 2^(G_i - G_j) is the product 2^(G_i - G_e) 2^(G_e - G_j) with e the last token of j's block
// of 16: a row factor for each block and a column factor.  Both are at most 1 where the block
// ends before i; in i's own block the first is not, and where a block decays by more than
// 2^-100 (an f32 product could under- or overflow) the pairs near the diagonal are
// computed one by one.
//
// Rows past the end of a sequence hold the next one's tokens (or TMA's zeros).  They are
// masked where they are a row or a column of P, and zeroed in shared memory where they are
// summed over (V and K): a zero factor would not do, 0 x NaN is NaN.
#include <cuda_runtime.h>
#include <stddef.h>

#include <algorithm>
#include <cmath>

#include "decay.cuh"
#include "ptx.cuh"

namespace gdn {
namespace {

constexpr int C = kDecayChunk;
constexpr int D = kHeadDim;
static_assert(C == 128 && D == 128, "the layouts below are those of 128 x 128 tiles");

// ------------------------------------------------------------ TMEM (columns)
constexpr uint32_t kTmAcc = 0;     // Q K^T (128), then P as packed pairs
constexpr uint32_t kTmO = 128;     // Q S^T, then the output
constexpr uint32_t kTmS = 256;     // S, f32 (128)
constexpr uint32_t kTmQ = 384;     // Q as packed pairs (64)
// P takes 16 columns for a block of 32 tokens: the first two blocks in front, the last two behind, so
// that a block goes over columns that its own warps have read.
__device__ __forceinline__ uint32_t p_block_col(int jb) { return kTmAcc + 16 * jb + (jb >= 2 ? 64 : 0); }
// V_d terms as packed pairs, in slots of up to 64 columns: one of its own, one over Q, which is free
// from Q S^T to the next chunk's copy, and one between the blocks of P.  A launch that makes states
// alone has the columns of the scores and the output for four.
constexpr uint32_t kTmVd = 448;
template <bool kStates>
__host__ __device__ constexpr int vd_slots() { return kStates ? 4 : 3; }
template <bool kStates>
__device__ __forceinline__ uint32_t vd_slot_col(int slot) {
  return kStates ? kTmAcc + 64 * slot : slot == 0 ? kTmVd : slot == 1 ? kTmQ : kTmAcc + 32;
}
constexpr uint32_t kTmCols = 512;
// kWide (a launch that meets f32 states): TMEM holds what one chunk adds, and the state itself is in the registers
// of warps 12-15, where each chunk is added to it in f32.  The tensor cores cut their sums off towards zero: with
// the state in TMEM each product of 16 tokens costs it half a unit in the last place, 1.8e-5 of a state of 16000 tokens
// and 7e-5 after 60000, which 16-bit states do not show; like this 5e-7, which is what the sum over a chunk costs.
// Where only states are made there is room for two chunks.  With the state in TMEM: 16 x 4096 with f32 states
// 385 us instead of 407, 2 x 65536 970 instead of 1055, 1024 short prompts 821 instead of 857, 256 tokens 12.7 instead of 13.0.
template <bool kWide>
__host__ __device__ constexpr bool apart() { return kWide; }
template <bool kStates>
__device__ __forceinline__ uint32_t sum_col(int ci) { return kStates ? kTmS + 128 * (ci & 1) : kTmS; }

// ------------------------------------------------------------ shared memory (bytes)
constexpr uint32_t kTile = C * D * 2;       // a 16-bit tile: two 128B-swizzled halves of 64 columns
constexpr uint32_t kHalf = kTile / 2;
constexpr uint32_t kOffKv = kTile;           // after Q: two stages of K, V; a launch that makes states
                                             // alone has a third over what follows
constexpr uint32_t kOffS = kOffKv + 4 * kTile;  // 16-bit copy of S
constexpr uint32_t kOffO = kOffS + kTile;    // the output tile on its way out
constexpr uint32_t kOffSmall = kOffO + kTile;
constexpr int kRecs = 3;
constexpr int kPoWarps = 8, kSWarps = 4, kVWarps = 8;
// f16 and a state that is kept apart: V_d is multiplied by powers of two (v_scale), the decays d by 2^kDExp
template <bool F16, bool kWide>
__host__ __device__ constexpr bool lifted() { return F16 && apart<kWide>(); }
constexpr int kDExp = 13;

struct Rec {       // one unit: a sequence, or a segment of one, of one head.  Only units with chunks go round
  int32_t t0, len, h, nch;  // first token, tokens, head, chunks (-1: no more units; h counts those without chunks)
  int32_t slot;     // in the pools (2^31 slots would be 64 TB)
  int32_t in, out;  // where the state comes from and goes to: a block of the workspace, or
};
constexpr int kPool = -1, kNone = -2;  // the caller's pool (zeros without one), or nowhere (zeros)
template <bool kStates>
__host__ __device__ constexpr int kv_stages() { return kStates ? 3 : 2; }
template <bool kStates, bool kInline_>
struct Small {
  static constexpr bool kInline = kInline_;  // slow waits
  float G[2][C];   // inclusive prefix sums of log2 g
  float d[2][C];   // 2^(sum of the log2 g behind the token), 0 past the end; with two V_d terms
                   // as 16-bit halves, C high ones and C low ones
  float cf[kStates ? 4 : C];  // 2^(G_e - G_j), e the last token of j's block of 16
  int32_t mild[2]; // no block of 16 tokens decays by more than 2^-100
  float gamma[2];  // 2^(G_last); where the state is kept apart and the decay is slow, 2^(G_last) - 1 with the sign bit set
  alignas(16) uint32_t claim[4];  // the answer to a claim of another unit
  int8_t v_exp[4][kVWarps];  // what the 16 values of each warp of V_d add is 2^v_exp times too large (the last four chunks)
  Rec rec[kRecs];
  uint64_t q_full, q_empty, k_full[kv_stages<kStates>()], v_full[kv_stages<kStates>()], kv_empty[kv_stages<kStates>()];
  uint64_t rec_full[kRecs], rec_empty[kRecs], claim_full;
  uint64_t gate_full[2], gate_empty[2], cf_empty;
  union {
    struct { uint64_t qk_done, qs_done, s_done, o_done; };  // products that have completed
    struct { uint64_t sum_done[2], sum_free[2]; };          // where only states are made: what a chunk adds
  };
  uint64_t q_ready, p_ready, o_free, o_staged;  // warps 4-11
  uint64_t o_stored, f_half, f_stored;          // warp 3
  uint64_t f_staged, si_full;                   // warps 12-15; an incoming 16-bit state
  uint64_t sf_full, sf_empty;                   // an incoming f32 state
  uint64_t s_ready, vd_full[vd_slots<kStates>()];  // warps 12-15, 16-23
  uint64_t vd_empty[vd_slots<kStates>()], drain;
  uint32_t tmem;
  int32_t abort, tries;  // side by side: wait_slow takes the address of the first
};
constexpr uint32_t kSmem = kOffSmall + std::max({sizeof(Small<false, false>), sizeof(Small<false, true>), sizeof(Small<true, true>)});
static_assert(kSmem <= 227 * 1024, "shared memory budget");

constexpr int kThreads = 32 * (4 + kPoWarps + kSWarps + kVWarps);
// Registers a thread: what a launch has, and how a launch that keeps the state apart shares them out among its
// groups of four warps.  The state needs 216 to stay without spills: with 200 the long cases take 1 to 2 % more,
// 1024 short prompts with f32 states 10 %.
constexpr int kRegs = 80, kRegsOne = 56, kRegsPo = 56, kRegsState = 216, kRegsV = 48;
static_assert(4 * kRegsOne + kPoWarps * kRegsPo + kSWarps * kRegsState + kVWarps * kRegsV <= kThreads / 32 * kRegs, "registers of a launch");
// The stages of K and V as a role goes through them, with the phase of each.
template <bool kStates>
struct Ring {
  int s = 0;
  uint32_t phases = 0;
  __device__ __forceinline__ uint32_t phase() const { return phases >> s & 1; }
  __device__ __forceinline__ void pass() { s = s + 1 == kv_stages<kStates>() ? 0 : s + 1; }  // over an f32 state
  __device__ __forceinline__ void next() { phases ^= 1u << s; pass(); }                      // over a chunk
};

// Every wait: bounded (0.2 s in probes of kProbeNs, or kProbeInlineNs), and over as soon as another
// role has given up.  Only the first probe is in line: the roles together fill the instruction cache.  Where the
// groups of warps share registers out among them there can be no call, and a single loop in line is the smallest.
constexpr uint64_t kWaitNs = 200000000, kProbeNs = 4000, kProbeInlineNs = 1400;
__device__ __noinline__ bool wait_slow(const volatile int32_t* abort, uint64_t* bar, uint32_t parity) {
  bool ok = false;
#pragma unroll 1
  for (int left = abort[1]; left > 0 && !ok && !*abort; --left) ok = mbar_try_wait_sleep(bar, parity, 20000u);
  return __all_sync(0xffffffffu, ok);
}
template <class Sm>
__device__ __forceinline__ bool wait(Sm* sm, uint64_t* bar, uint32_t parity) {
  if (Sm::kInline) {
    int left = sm->tries;
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
      if (--left == 0 || *reinterpret_cast<const volatile int32_t*>(&sm->abort)) return false;
    return true;
  }
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_slow(&sm->abort, bar, parity);
}
// The same for copies and products under way when a CTA ends, whoever gave up.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (uint64_t ns = 0; ns < kWaitNs && !mbar_try_wait_sleep(bar, parity, 20000u); ns += kProbeNs) {}
}
template <class Sm>
__device__ __forceinline__ void give_up(const DecayPrefillParams& p, Sm* sm) {
  *reinterpret_cast<volatile int32_t*>(&sm->abort) = 1;
  atomicOr(p.dev_err, kDevErrTimeout);
}
// One arrival for the warp, behind everything its lanes have done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The next unit's record, for every role but the producer; false when there is none left
// or a wait gave up (*failed).
template <class Sm>
__device__ __forceinline__ bool next_unit(Sm* sm, int u, int lane, Rec* r, bool* failed) {
  const int slot = u % kRecs;
  if (!wait(sm, &sm->rec_full[slot], (u / kRecs) & 1)) {
    *failed = true;
    return false;
  }
  *r = sm->rec[slot];
  warp_arrive(&sm->rec_empty[slot], lane);
  return r->nch >= 0;
}

// ------------------------------------------------------------ units
// kStates, here and below: the launch makes the states that the segments add, no outputs.  It walks a
// segment from its last chunk to its first: with decays counted to the end of the segment, V_d^T K
// of all chunks just adds up.
template <bool kStates>
__device__ __forceinline__ int64_t unit_count(const DecayPrefillParams& p) {
  return (int64_t)p.N * (kStates ? p.splits - 1 : p.splits) * p.H;
}
// Unit x of the launch; device error bits instead where its bounds or its slot are bad.
template <bool kStates>
__device__ __forceinline__ int unit_at(const DecayPrefillParams& p, int64_t x, Rec* r) {
  // heads of a segment side by side: they share keys and queries, or lines of the gates
  const int segs = kStates ? p.splits - 1 : p.splits;
  const int h = (int)(x % p.H), seg = (int)(x / p.H) % segs, n = (int)(x / p.H / segs);
  const int64_t bos = index_at(p.cu, p.cu_dtype, n), eos = index_at(p.cu, p.cu_dtype, n + 1);
  const int64_t slot = p.state_idx ? index_at(p.state_idx, p.idx_dtype, n) : (int64_t)n;
  int err = 0;
  if (bos < 0 || eos < bos || eos > p.T) err |= kDevErrCu;
  if ((p.s_in && (slot < 0 || slot >= p.sin_slots)) || (p.s_out && (slot < 0 || slot >= p.sout_slots))) err |= kDevErrIdx;
  if (err) return err;
  const int all = (int)((eos - bos + C - 1) / C);  // chunks of the sequence
  const int c0 = (int)((int64_t)all * seg / p.splits), nch = (int)((int64_t)all * (seg + 1) / p.splits) - c0;
  const int first = (int)bos + c0 * C, len = nch > 0 ? min((int)eos - first, nch * C) : 0;
  const int block = (n * p.H + h) * (p.splits - 1) + seg;  // of the state behind this segment
  *r = Rec{first, len, h, nch, (int)slot, seg == 0 ? kPool : kStates ? kNone : block - 1,
           kStates ? block : seg == p.splits - 1 ? kPool : kNone};
  return 0;
}

// Whether a unit's state comes by TMA, in 16 bits straight into the place of its 16-bit copy or in f32
// into a stage of K and V (as those behind segments do), and whether the one that it leaves goes by
// TMA, from the place of the copy: f32 in two halves of 64 columns.
// kWide: a launch that meets f32 states; the others keep the instructions for them out of the cache.
template <bool kWide>
__device__ __forceinline__ bool state_in_tma(const DecayPrefillParams& p, const Rec& r) {
  return p.sin_tma && r.in == kPool && !(kWide && p.sin_dtype == kF32);
}
template <bool kWide>
__device__ __forceinline__ bool state_in_ring(const DecayPrefillParams& p, const Rec& r) {
  if (!kWide) return false;
  return r.in >= 0 || (p.sin_tma && r.in == kPool && p.sin_dtype == kF32);
}
__device__ __forceinline__ bool state_out_tma(const DecayPrefillParams& p, const Rec& r) { return p.sout_tma && r.out == kPool; }
template <bool kWide>
__device__ __forceinline__ int state_out_parts(const DecayPrefillParams& p) { return kWide && p.sout_dtype == kF32 ? 2 : 1; }

// The state of a unit without chunks from where it comes to where it goes, by one warp.
template <bool kStates>
__device__ __forceinline__ void pass_on(const DecayPrefillParams& p, int h, int64_t slot, int in, int out, int lane) {
  if (kStates && lane == 0) p.ws_decay[out] = 1.f;
  if (out == kNone || (out == kPool && !p.s_out)) return;
  const bool pool = in == kPool && p.s_in;
  const int from_dtype = pool ? p.sin_dtype : kF32, to_dtype = out >= 0 ? kF32 : p.sout_dtype;
  const char* from = pool ? reinterpret_cast<const char*>(p.s_in) + (slot * p.sin_slot + (int64_t)h * p.sin_head) * (from_dtype == kF32 ? 4 : 2)
                          : in >= 0 ? reinterpret_cast<const char*>(p.ws + (int64_t)in * (D * D)) : nullptr;
  char* to = out >= 0 ? reinterpret_cast<char*>(p.ws + (int64_t)out * (D * D))
                        : reinterpret_cast<char*>(p.s_out) + (slot * p.sout_slot + (int64_t)h * p.sout_head) * (to_dtype == kF32 ? 4 : 2);
  constexpr int kBatch = 4;
#pragma unroll 1
  for (int e0 = 4 * lane; e0 < D * D; e0 += 128 * kBatch) {
    float2 x[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = e0 + 128 * i;
      x[i][0] = x[i][1] = make_float2(0.f, 0.f);
      if (!from) continue;
      if (from_dtype == kF32) {
        const float4 f = reinterpret_cast<const float4*>(from)[e / 4];
        x[i][0] = make_float2(f.x, f.y);
        x[i][1] = make_float2(f.z, f.w);
      } else {
        const uint2 f = reinterpret_cast<const uint2*>(from)[e / 4];
        x[i][0] = from_dtype == kF16 ? unpack16<true>(f.x) : unpack16<false>(f.x);
        x[i][1] = from_dtype == kF16 ? unpack16<true>(f.y) : unpack16<false>(f.y);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = e0 + 128 * i;
      if (to_dtype == kF32)
        reinterpret_cast<float4*>(to)[e / 4] = make_float4(x[i][0].x, x[i][0].y, x[i][1].x, x[i][1].y);
      else if (to_dtype == kF16)
        reinterpret_cast<uint2*>(to)[e / 4] = make_uint2(pack16x2<true>(x[i][0]), pack16x2<true>(x[i][1]));
      else
        reinterpret_cast<uint2*>(to)[e / 4] = make_uint2(pack16x2<false>(x[i][0]), pack16x2<false>(x[i][1]));
    }
  }
}

// ------------------------------------------------------------ warp 0: loads
template <bool kStates, bool kWide, bool kClaim, class Sm>
__device__ __forceinline__ void run_producer(const DecayPrefillParams& p, uint8_t* base, Sm* sm, int lane) {
  bool ok = true;
  int u = 0, ci = 0;  // units and chunks so far
  Ring<kStates> ring;
  uint32_t chunks_in = 0;  // bit s: a chunk has been in stage s
  int f32_stage = -1;      // the stage that holds an f32 state
  const int64_t units = unit_count<kStates>(p);
  int empties = 0;
  int q_loads = 0, s_loads = 0, sf_loads = 0, outs = 0;  // outs: states that the units so far leave by TMA
  auto stage_free = [&] {
    const int s = ring.s;
    if (s == f32_stage) {
      f32_stage = -1;
      return wait(sm, &sm->sf_empty, (sf_loads - 1) & 1);
    }
    return !(chunks_in >> s & 1) || wait(sm, &sm->kv_empty[s], ring.phase() ^ 1);
  };
  auto publish = [&](const Rec& r) {
    const int slot = u % kRecs;
    if (u >= kRecs && !wait(sm, &sm->rec_empty[slot], (u / kRecs - 1) & 1)) return false;
    if (lane == 0) {
      sm->rec[slot] = r;
      mbar_arrive(&sm->rec_full[slot]);
    }
    ++u;
    return true;
  };
  // The first unit is that of the CTA's place in the grid.  Then, with a grid of one CTA an SM, every
  // gridDim.x-th one; or, with a CTA for each unit, those of CTAs that have not been launched, taken over
  // one at a time when the last chunk of the one before is loaded.
  int64_t x = blockIdx.x;
  int claims = 0;
  auto claim = [&] {
    if (!kClaim) return;
    __syncwarp();
    if (lane == 0) {
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&sm->claim_full, 16);
      clc_ask(sm->claim, &sm->claim_full);
    }
    ++claims;
  };
  auto another = [&] {
    if (!kClaim) return (x += gridDim.x) < units;
    uint32_t to = 0;
    ok = wait(sm, &sm->claim_full, (claims - 1) & 1);
    const bool any = ok && clc_answer(sm->claim, &to);
    x = to;
    return any;
  };
  for (bool more = true; more; more = ok && another()) {
    Rec r;
    const int err = unit_at<kStates>(p, x, &r);
    if (err || r.nch == 0) claim();
    if (err) {
      if (lane == 0) atomicOr(p.dev_err, err);
      continue;
    }
    if (r.nch == 0) {  // nothing but a state to pass on: warps 12-15 see to these at the end, if they can find them
      if (kClaim) pass_on<kStates>(p, r.h, r.slot, r.in, r.out, lane);
      else ++empties;
      continue;
    }
    ok = publish(r);
    if (!ok) break;
    const int h = r.h, nch = r.nch, first = r.t0;
    if (!kStates && state_in_ring<kWide>(p, r)) {
      ok = stage_free();
      if (!ok) break;
      if (lane == 0) {
        uint8_t* dst = base + kOffKv + ring.s * 2 * kTile;
        mbar_arrive_expect_tx(&sm->sf_full, 2 * kTile);
        for (int q = 0; q < 4; ++q)
          if (r.in >= 0) tma_load_4d(dst + q * kHalf, &p.tm_ws, &sm->sf_full, 32 * q, 0, 0, r.in);
          else tma_load_4d(dst + q * kHalf, &p.tm_sin, &sm->sf_full, 32 * q, 0, r.h, r.slot);
      }
      ++sf_loads;
      f32_stage = ring.s;
      ring.pass();
    } else if (p.s_in && r.in == kPool && lane == 0) {
      const int es = p.sin_dtype == kF32 ? 4 : 2;
      bulk_prefetch_l2(reinterpret_cast<const char*>(p.s_in) + ((int64_t)r.slot * p.sin_slot + (int64_t)h * p.sin_head) * es, D * D * es);
    }
    const int hq = h / (p.H / p.H_qk), hv = h / (p.H / p.H_v);
    for (int c = 0; c < nch; ++c, ++ci) {
      if (c + 1 == nch) claim();
      const int s = ring.s, t0 = first + (kStates ? nch - 1 - c : c) * C;
      auto load = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* bar, int head) {
        mbar_arrive_expect_tx(bar, kTile);
        tma_load_3d(dst, tm, bar, 0, head, t0);
        tma_load_3d(dst + kHalf, tm, bar, 64, head, t0);
      };
      if (!kStates) {
        ok = ci < 1 || wait(sm, &sm->q_empty, (ci - 1) & 1);
        if (!ok) break;
        if (lane == 0) load(base, &p.tm_q, &sm->q_full, hq);
        ++q_loads;
      }
      ok = stage_free();
      if (!ok) break;
      chunks_in |= 1u << s;
      if (lane == 0) {
        uint8_t* k = base + kOffKv + s * 2 * kTile;
        load(k, &p.tm_k, &sm->k_full[s], hq);
        load(k + kTile, &p.tm_v, &sm->v_full[s], hv);
      }
      ring.next();
      if (!kStates && c == 0 && state_in_tma<kWide>(p, r)) {
        // what was in its place has been read: by Q S^T, by warps 12-15, and by the state's own way out
        ok = (ci == 0 || (wait(sm, &sm->qs_done, (ci - 1) & 1) && wait(sm, &sm->s_ready, (ci - 1) & 1))) &&
             (outs == 0 || wait(sm, &sm->f_stored, (outs - 1) & 1));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm->si_full, kTile);
          tma_load_4d(base + kOffS, &p.tm_sin, &sm->si_full, 0, 0, h, r.slot);
          tma_load_4d(base + kOffS + kHalf, &p.tm_sin, &sm->si_full, 64, 0, h, r.slot);
        }
        ++s_loads;
      }
    }
    if (!kStates && state_out_tma(p, r)) ++outs;
  }
  if (ok) ok = publish(Rec{0, 0, empties, -1, 0, 0, 0});
  if (!ok && lane == 0) give_up(p, sm);
  // loads that no role waits for any more land before the CTA's shared memory goes away
  for (int s = 0; s < kv_stages<kStates>(); ++s) {
    if (!(chunks_in >> s & 1)) continue;
    drain(&sm->k_full[s], (ring.phases >> s & 1) ^ 1);
    drain(&sm->v_full[s], (ring.phases >> s & 1) ^ 1);
  }
  if (claims) drain(&sm->claim_full, (claims - 1) & 1);
  if (q_loads) drain(&sm->q_full, (q_loads - 1) & 1);
  if (s_loads) drain(&sm->si_full, (s_loads - 1) & 1);
  if (sf_loads) drain(&sm->sf_full, (sf_loads - 1) & 1);
}

// ------------------------------------------------------------ warp 1: products
// V_d is made in parts of kSub tokens, kSub / 2 columns a term: two of 64 tokens in slots 0 and 1, or,
// with three terms, four of 32 in slots 0, 1, 0 and 2.
template <int kTerms>
__host__ __device__ constexpr int sub_tokens() { return kTerms == 2 ? 64 : 32; }
// Where only states are made, each part has a slot.
template <int kTerms, bool kStates>
__device__ __forceinline__ void vd_place(int ci, int b, int* slot, int* round) {  // round: uses of the slot before
  *slot = kTerms == 2 || kStates ? b : b == 3 ? 2 : b & 1;
  *round = kTerms == 3 && !kStates && *slot == 0 ? 2 * ci + (b >> 1) : ci;
}

template <bool F16, int kTerms, bool kStates, bool kWide, class Sm>
__device__ __forceinline__ void run_mma(const DecayPrefillParams& p, uint8_t* base, Sm* sm, uint32_t tmem, int lane) {
  constexpr int kSub = sub_tokens<kTerms>(), kSubs = C / kSub;
  const uint32_t id_kk = idesc_16_f32(F16, 128, 128, 0, 0, 0);  // B K-major
  const uint32_t id_kmn = idesc_16_f32(F16, 128, 128, 0, 1, 0); // B MN-major (its rows are summed over)
  const uint32_t id_kmn_neg = idesc_16_f32(F16, 128, 128, 0, 1, 1);  // the first of two V_d terms is stored negated
  const uint64_t d_s = sdesc_sw128(smem_u32(base + kOffS), 16, 1024);
  const bool leader = elect_one();
  bool failed = false;
  Rec r;
  int ci = 0, ins = 0;  // chunks so far; 16-bit states by TMA
  Ring<kStates> ring;
  for (int u = 0; next_unit(sm, u, lane, &r, &failed); ++u) {
    if (!kStates && state_in_ring<kWide>(p, r)) ring.pass();
    for (int c = 0; c < r.nch; ++c, ++ci, ring.next()) {
      const int s = ring.s;
      const uint32_t ph = ring.phase(), one = ci & 1;
      const uint32_t k = smem_u32(base + kOffKv + s * 2 * kTile);
      const uint64_t d_k = sdesc_sw128(k, 16, 1024), d_kt = sdesc_sw128(k, kHalf, 1024);
      const uint64_t d_vt = sdesc_sw128(k + kTile, kHalf, 1024);
      if (kStates) {  // what the chunk before the last added has been read
        if (!(wait(sm, &sm->k_full[s], ph) && (ci < 2 || wait(sm, &sm->sum_free[one], ((ci >> 1) - 1) & 1)))) { failed = true; break; }
      } else {
        // Q K^T.  P of the chunk before is being read by its P V at the latest, which was
        // issued before: the products run in order.
        if (!(wait(sm, &sm->k_full[s], ph) && wait(sm, &sm->q_ready, one))) { failed = true; break; }
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mma_ts(tmem + kTmAcc, tmem + kTmQ + i * 8, d_k + ((i >> 2) * kHalf + (i & 3) * 32) / 16, id_kk, i > 0);
          mma_commit(&sm->qk_done);
        }
        __syncwarp();
        // Q S^T
        const bool direct = c == 0 && state_in_tma<kWide>(p, r);  // the copy that is read came by TMA
        if (!((direct ? wait(sm, &sm->si_full, ins & 1) : wait(sm, &sm->s_ready, one)) &&
              (ci == 0 || wait(sm, &sm->o_free, one ^ 1)))) { failed = true; break; }
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mma_ts(tmem + kTmO, tmem + kTmQ + i * 8, d_s + ((i >> 2) * kHalf + (i & 3) * 32) / 16, id_kk, i > 0);
          mma_commit(&sm->qs_done);
        }
        __syncwarp();
        if (direct) {
          ++ins;
          if (!wait(sm, &sm->s_ready, one)) { failed = true; break; }
        }
      }
      // V_d^T K
#pragma unroll 1
      for (int b = 0; b < kSubs; ++b) {
        int slot, round;
        vd_place<kTerms, kStates>(ci, b, &slot, &round);
        if (!wait(sm, &sm->vd_full[slot], round & 1)) { failed = true; break; }
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int t = 0; t < kTerms; ++t)
#pragma unroll
            for (int i = 0; i < kSub / 16; ++i)
              mma_ts(tmem + sum_col<kStates>(ci), tmem + vd_slot_col<kStates>(slot) + t * (kSub / 2) + i * 8, d_kt + (b * (kSub / 16) + i) * 128,
                     kTerms == 2 && t == 0 ? id_kmn_neg : id_kmn, !apart<kWide>() || b + t + i > 0);
          mma_commit(&sm->vd_empty[slot]);
          if (b == kSubs - 1) mma_commit(kStates ? &sm->sum_done[one] : &sm->s_done);
          if (kStates && b == kSubs - 1) mma_commit(&sm->kv_empty[s]);
        }
        __syncwarp();
      }
      if (failed) break;
      if (kStates) continue;
      // + P V
      if (!wait(sm, &sm->p_ready, one)) { failed = true; break; }
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          mma_ts(tmem + kTmO, tmem + p_block_col(i / 2) + (i & 1) * 8, d_vt + i * 128, id_kmn, 1);
        mma_commit(&sm->o_done);
        mma_commit(&sm->kv_empty[s]);
      }
      __syncwarp();
    }
    if (failed) break;
  }
  if (failed && lane == 0) give_up(p, sm);
  if (leader) mma_commit(&sm->drain);
  __syncwarp();
  drain(&sm->drain, 0);  // no product is under way when TMEM is freed
}

// ------------------------------------------------------------ warp 2: gates
template <bool F16, int kTerms, bool kStates, bool kWide, class Sm>
__device__ __forceinline__ void run_gates(const DecayPrefillParams& p, Sm* sm, int lane) {
  bool failed = false;
  Rec r{};
  int ci = 0;
  // this lane's four gates of chunk c (1 past the end): the loads of a dtype go out together,
  // and a chunk ahead of their use
  auto load4 = [&](int c, float (&g)[4]) {
    const int64_t at = ((int64_t)r.t0 + c * C + 4 * lane) * p.g_st + (int64_t)r.h * p.g_sh;
    const int left = r.len - c * C - 4 * lane;
    auto each = [&](auto conv) {
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = e < left ? conv(at + e * p.g_st) : 1.f;
    };
    if (p.g_dtype == kF32) each([&](int64_t i) { return reinterpret_cast<const float*>(p.g)[i]; });
    else if (p.g_dtype == kBF16) each([&](int64_t i) { return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.g)[i]); });
    else each([&](int64_t i) { return __half2float(reinterpret_cast<const __half*>(p.g)[i]); });
  };
  for (int u = 0; next_unit(sm, u, lane, &r, &failed); ++u) {
    float ahead[4] = {1.f, 1.f, 1.f, 1.f}, later = 0.f;  // later: the decay behind this chunk (states)
    auto chunk_at = [&](int c) { return kStates ? r.nch - 1 - c : c; };
    if (p.g && r.nch > 0) load4(chunk_at(0), ahead);
    for (int c = 0; c < r.nch; ++c, ++ci) {
      const int b = ci & 1, left = r.len - chunk_at(c) * C;
      float lg[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) lg[e] = log2f(fminf(fmaxf(ahead[e], FLT_MIN), 1.f));
      if (p.g && c + 1 < r.nch) load4(chunk_at(c + 1), ahead);
      // prefix and suffix sums: the suffix is summed on its own, since G_last - G_j would
      // carry the rounding of two large sums into the state
      float pre[4], suf[4];
      pre[0] = lg[0]; pre[1] = pre[0] + lg[1]; pre[2] = pre[1] + lg[2]; pre[3] = pre[2] + lg[3];
      suf[3] = 0.f; suf[2] = lg[3]; suf[1] = suf[2] + lg[2]; suf[0] = suf[1] + lg[1];
      float up = pre[3], down = pre[3];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float a = __shfl_up_sync(0xffffffffu, up, o), z = __shfl_down_sync(0xffffffffu, down, o);
        if (lane >= o) up += a;
        if (lane + o < 32) down += z;
      }
      float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
      if (lane == 0) before = 0.f;
      if (lane == 31) behind = 0.f;
      if (kStates) behind += later;
      const float total = __shfl_sync(0xffffffffu, down, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) { pre[e] += before; suf[e] += behind; }
      const float g_end = __shfl_sync(0xffffffffu, pre[3], lane | 3);  // the last token of the block of 16
      const float g_begin = __shfl_sync(0xffffffffu, before, lane & ~3);
      const bool mild = __all_sync(0xffffffffu, g_begin - g_end <= 100.f);
      if (!(ci < 2 || wait(sm, &sm->gate_empty[b], ((ci >> 1) - 1) & 1))) { failed = true; break; }
      *reinterpret_cast<float4*>(&sm->G[b][4 * lane]) = make_float4(pre[0], pre[1], pre[2], pre[3]);
      float d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = 4 * lane + e < left ? exp2f(suf[e]) * (lifted<F16, kWide>() ? float(1 << kDExp) : 1.f) : 0.f;
      if (kTerms == 2) {
        uint32_t* dh = reinterpret_cast<uint32_t*>(sm->d[b]) + 2 * lane;
        const uint32_t h0 = pack16x2<F16>(d[0], d[1]), h1 = pack16x2<F16>(d[2], d[3]);
        const float2 f0 = unpack16<F16>(h0), f1 = unpack16<F16>(h1);
        *reinterpret_cast<uint2*>(dh) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(dh + C / 2) = make_uint2(pack16x2<F16>(d[0] - f0.x, d[1] - f0.y), pack16x2<F16>(d[2] - f1.x, d[3] - f1.y));
      } else {
        *reinterpret_cast<float4*>(&sm->d[b][4 * lane]) = make_float4(d[0], d[1], d[2], d[3]);
      }
      if (lane == 0) {
        // b S + a S with a = 2^(G_last) - 1 knows a decay near 1 far better than 2^(G_last) S, whose error is the same
        // one in every chunk of equal gates
        const bool slow = apart<kWide>() && total > -1.f;
        sm->gamma[b] = slow ? copysignf(expm1f(total * 0.693147180559945f), -1.f) : exp2f(total);
        sm->mild[b] = mild;
      }
      later += total;
      if (kStates && c + 1 == r.nch && lane == 0) p.ws_decay[r.out] = exp2f(later);
      if (!kStates) {
        if (!(ci == 0 || wait(sm, &sm->cf_empty, (ci - 1) & 1))) { failed = true; break; }
        *reinterpret_cast<float4*>(&sm->cf[4 * lane]) = make_float4(
            exp2_fast(g_end - pre[0]), exp2_fast(g_end - pre[1]), exp2_fast(g_end - pre[2]), exp2_fast(g_end - pre[3]));
      }
      warp_arrive(&sm->gate_full[b], lane);
    }
    if (failed) break;
  }
  if (failed && lane == 0) give_up(p, sm);
}

// ------------------------------------------------------------ warp 3: output stores
template <bool kWide, class Sm>
__device__ __forceinline__ void run_store(const DecayPrefillParams& p, uint8_t* base, Sm* sm, int lane) {
  bool failed = false;
  Rec r;
  int ci = 0, outs = 0;  // tiles and parts of states that have gone out
  for (int u = 0; next_unit(sm, u, lane, &r, &failed); ++u) {
    for (int c = 0; c < r.nch; ++c, ++ci) {
      const int t0 = r.t0 + c * C, left = r.len - c * C;
      if (c + 1 == r.nch && state_out_tma(p, r)) {  // ready before the last tile is
        const int parts = state_out_parts<kWide>(p), cols = 64 / parts;
        for (int x = 0; x < parts && !failed; ++x) {
          if (!wait(sm, &sm->f_staged, outs++ & 1)) { failed = true; break; }
          if (lane == 0) {
            tma_store_4d(&p.tm_sout, base + kOffS, 64 * x, 0, r.h, r.slot);
            tma_store_4d(&p.tm_sout, base + kOffS + kHalf, 64 * x + cols, 0, r.h, r.slot);
            bulk_commit();
            bulk_wait_read_all();
          }
          warp_arrive(x + 1 < parts ? &sm->f_half : &sm->f_stored, lane);
        }
        if (failed) break;
      }
      if (!wait(sm, &sm->o_staged, ci & 1)) { failed = true; break; }
      uint8_t* tile = base + kOffO;
      if (left >= C) {
        if (lane == 0) {
          tma_store_3d(&p.tm_o, tile, 0, r.h, t0);
          tma_store_3d(&p.tm_o, tile + kHalf, 64, r.h, t0);
          bulk_commit();
          bulk_wait_read_all();
        }
      } else {  // only the sequence's own rows: the next rows belong to another unit
        const int ch = lane & 15;
        const uint8_t* from = tile + (ch >> 3) * kHalf;
        char* o = reinterpret_cast<char*>(p.out) + ((int64_t)(t0 + (lane >> 4)) * p.o_st + (int64_t)r.h * p.o_sh) * 2 + ch * 16;
#pragma unroll 4
        for (int row = lane >> 4; row < left; row += 2, o += p.o_st * 4)
          *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(from + sw128_chunk(row, ch & 7));
      }
      warp_arrive(&sm->o_stored, lane);
    }
    if (failed) break;
  }
  if (failed && lane == 0) give_up(p, sm);
  if (lane == 0) bulk_wait_read_all();
}

// ------------------------------------------------------------ warps 4-11: P and the output
template <bool F16, bool kWide, class Sm>
__device__ __forceinline__ void run_po(const DecayPrefillParams& p, uint8_t* base, Sm* sm, uint32_t tmem, int warp, int lane) {
  const int w = warp & 3, hf = (warp >> 2) - 1, row = 32 * w + lane;  // warps 4-11: columns 0 .. 63, 8-11: 64 .. 127
  const uint32_t tr = tmem + ((uint32_t)(32 * w) << 16);
  bool failed = false;
  Rec r;
  int u = 0, left = 0;  // units seen, chunks of the current one that are not begun
  auto another = [&] {  // whether there is a chunk to begin
    if (left == 0 && next_unit(sm, u, lane, &r, &failed)) { left = r.nch; ++u; }
    return left-- > 0;
  };
  // Q of chunk `at` from shared memory to TMEM, the A operand of two products, once V_d^T K of the
  // chunk before has read the V_d that took its place.
  const uint32_t qa = smem_u32(base);
  auto copy_q = [&](int at) {
    if (!(wait(sm, &sm->q_full, at & 1) && (at == 0 || wait(sm, &sm->s_done, (at - 1) & 1)))) return false;
    tc_fence_after();
    const int rr = 32 * w + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll 2
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int rb = 0; rb < 2; ++rb) {
        const int i = 4 * hf + j, ch = 2 * i + (lane >> 4);
        uint32_t a[4];
        ldmatrix_x4(qa + (ch >> 3) * kHalf + sw128_chunk(rr + 16 * rb, ch & 7), a);
        tmem_st16x128_x2(tr + ((uint32_t)(16 * rb) << 16) + kTmQ + 8 * i, a);
      }
    tmem_st_wait();
    tc_fence_before();
    warp_arrive(&sm->q_ready, lane);
    if (lane == 0) mbar_arrive(&sm->q_empty);
    return true;
  };
  bool more = another();
  if (more && !copy_q(0)) failed = true;
  for (int ci = 0; more && !failed; ++ci) {
    {
      const int b = ci & 1;
      const uint32_t one = ci & 1;
      if (!(wait(sm, &sm->gate_full[b], (ci >> 1) & 1) && wait(sm, &sm->qk_done, one))) { failed = true; break; }
      tc_fence_after();
      const float gi = sm->G[b][row];
      const bool mild = sm->mild[b] != 0;
      // P in blocks of 16 columns, by factors up to this warp's diagonal ones and zeros behind them, in the
      // order 0 .. 3 and 7 .. 4 so that each goes over columns that its warp has read.  Rolled up: the
      // roles together fill the instruction cache.
#pragma unroll 1
      for (int it = 0; it < 4; ++it) {
        const int jb = hf ? 7 - it : it, j0 = 16 * jb;
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pk[e] = 0u;
        if (jb <= 2 * w + 1) {
          uint32_t x[16];
          tmem_ld16(tr + kTmAcc + j0, x);
          const float2 rf = pair(p.scale * exp2_fast(gi - sm->G[b][j0 + 15]));
          tmem_ld_wait();
          if (mild || jb < 2 * w) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float4 f = *reinterpret_cast<const float4*>(&sm->cf[j0 + 2 * e]);
              pk[e] = pack16x2<F16>(mul2(pair_at(x + 2 * e), mul2(make_float2(f.x, f.y), rf)));
              pk[e + 1] = pack16x2<F16>(mul2(pair_at(x + 2 * e + 2), mul2(make_float2(f.z, f.w), rf)));
            }
          } else {  // pair by pair
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 f = *reinterpret_cast<const float2*>(&sm->G[b][j0 + 2 * e]);
              pk[e] = pack16x2<F16>(mul2(mul2(pair_at(x + 2 * e), pair(p.scale)), make_float2(exp2_fast(gi - f.x), exp2_fast(gi - f.y))));
            }
          }
          if (jb >= 2 * w) {  // pairs behind the diagonal, whose factor may be infinite, go
            const int d = row - j0;
#pragma unroll
            for (int e = 0; e < 8; ++e) pk[e] = 2 * e > d ? 0u : 2 * e == d ? pk[e] & 0xffffu : pk[e];
          }
        }
        tmem_st8(tr + p_block_col(jb / 2) + 8 * (jb & 1), pk);
      }
      tc_fence_before();
      warp_arrive(&sm->cf_empty, lane);
      // Q S^T of the row times scale 2^G_i
      if (!wait(sm, &sm->qs_done, one)) { failed = true; break; }
      tc_fence_after();
      const float2 gam = pair(p.scale * exp2f(gi));
#pragma unroll 1
      for (int q = 2 * hf; q < 2 * hf + 2; ++q) {
        uint32_t a[32];
        tmem_ld32(tr + kTmO + 32 * q, a);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = mul2(pair_at(a + e), gam);
          a[e] = __float_as_uint(x.x);
          a[e + 1] = __float_as_uint(x.y);
        }
        tmem_st32(tr + kTmO + 32 * q, a);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&sm->p_ready, lane);
      if (lane == 0) mbar_arrive(&sm->gate_empty[b]);
      more = another();
      if (failed || (more && !copy_q(ci + 1))) { failed = true; break; }
      // the output tile, once the one before has left
      if (!(wait(sm, &sm->o_done, one) && (ci == 0 || wait(sm, &sm->o_stored, one ^ 1)))) { failed = true; break; }
      tc_fence_after();
      uint8_t* tile = base + kOffO;
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        uint32_t a[32];
        tmem_ld32(tr + kTmO + 64 * hf + 32 * q, a);
        tmem_ld_wait();
        if (q == 1) {
          tc_fence_before();
          warp_arrive(&sm->o_free, lane);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(tile + hf * kHalf + sw128_chunk(row, 4 * q + e)) =
              make_uint4(pack16x2<F16>(pair_at(a + 8 * e)), pack16x2<F16>(pair_at(a + 8 * e + 2)),
                         pack16x2<F16>(pair_at(a + 8 * e + 4)), pack16x2<F16>(pair_at(a + 8 * e + 6)));
      }
      fence_proxy_async_smem();
      warp_arrive(&sm->o_staged, lane);
    }
  }
  if (failed && lane == 0) give_up(p, sm);
}

// ------------------------------------------------------------ warps 12-15: the state
// 32 values of a state row, as the bits of f32.
template <bool kWide>
__device__ __forceinline__ void load_state32(const void* base, int dtype, int64_t off, uint32_t (&s)[32]) {
  if (kWide && dtype == kF32) {
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 x = q[i];
      s[4 * i] = x.x; s[4 * i + 1] = x.y; s[4 * i + 2] = x.z; s[4 * i + 3] = x.w;
    }
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = q[i];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = dtype == kF16 ? unpack16<true>(w[e]) : unpack16<false>(w[e]);
        s[8 * i + 2 * e] = __float_as_uint(f.x);
        s[8 * i + 2 * e + 1] = __float_as_uint(f.y);
      }
    }
  }
}
template <bool kWide>
__device__ __forceinline__ void store_state32(void* base, int dtype, int64_t off, const uint32_t (&s)[32]) {
  if (kWide && dtype == kF32) {
    uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
  } else {
    uint4* q = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = pair_at(s + 8 * i + 2 * e);
        w[e] = dtype == kF16 ? pack16x2<true>(f) : pack16x2<false>(f);
      }
      q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// a (d_hi + d_lo) for a pair of 16-bit values as lo - neg: neg is the rounded product of a and
// -d_hi, lo the rest of it (exact where f16 reaches down to it: a product of two 16-bit values has no more
// bits than two of them hold) plus the product of a and d_lo.
template <bool F16>
__device__ __forceinline__ void split_product(uint32_t a, uint32_t dh, uint32_t dl, uint32_t* neg, uint32_t* lo) {
  auto go = [&](auto x, auto h, auto mh, auto l) {
    const auto n = __hmul2(x, mh);
    const auto r = __hfma2(x, l, __hfma2(x, h, n));
    *neg = *reinterpret_cast<const uint32_t*>(&n);
    *lo = *reinterpret_cast<const uint32_t*>(&r);
  };
  uint32_t mh = dh ^ 0x80008000u;
  if (F16) go(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&dh), *reinterpret_cast<__half2*>(&mh), *reinterpret_cast<__half2*>(&dl));
  else go(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&dh), *reinterpret_cast<__nv_bfloat162*>(&mh), *reinterpret_cast<__nv_bfloat162*>(&dl));
}

// f16 does not reach far down: two terms hold 22 bits of products near 1, but of 1e-3 only 15.  So V_d of the 16 values
// of a warp goes times the power of two that brings the largest value to 2 .. 4 (and d to 2^kDExp), and warps 12-15 take
// it back when they add the chunk: an error of 2^-22 of the product, or 2^-39 of the largest value.  Values are
// made larger and never smaller, d the other way round, so that neither loses bits.  Values of 1e-3: 8e-5 -> 2e-7 of
// an f32 state; 16 x 4096 of 32 heads 348 -> 386 us, 32000
// tokens of 8 heads 3 % more.  (An f16 state does without: it has no more bits there than the two terms.)
__device__ __forceinline__ int v_scale(uint32_t va, int m, int lr, int ch) {  // log2
  __half2 most = __half2half2(__ushort_as_half(0));
#pragma unroll 2
  for (int tok = 0; tok < C; tok += 16) {
    uint32_t a[4];
    ldmatrix_x4_trans(va + sw128_chunk(tok + (m >> 1) * 8 + lr, ch & 7), a);
#pragma unroll
    for (int e = 0; e < 4; ++e) most = __hmax2(most, __habs2(*reinterpret_cast<const __half2*>(&a[e])));
  }
  const int e = (int)(__reduce_max_sync(0xffffffffu, (uint32_t)__half_as_ushort(__hmax(__low2half(most), __high2half(most)))) >> 10);
  return max(min(16 - e, 15), -14);
}

// Zero this warp's share of the rows past the end: 16 columns (two 16-byte chunks from ch0) of K, and of
// V, exactly what the warp reads below.  Of several groups each takes the rows of its own parts.
template <int kSub, int kGroups>
__device__ __forceinline__ void zero_tails(uint8_t* k, uint8_t* v, int left, int ch0, int group, int lane) {
  for (int e = 2 * left + lane; e < C * 2; e += 32) {
    if ((e >> 1) / kSub % kGroups != group) continue;
    const int ch = ch0 + (e & 1);
    const uint32_t at = (ch >> 3) * kHalf + sw128_chunk(e >> 1, ch & 7);
    *reinterpret_cast<uint4*>(k + at) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(v + at) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <bool F16, int kTerms, bool kStates, bool kWide, class Sm>
__device__ __forceinline__ void run_state(const DecayPrefillParams& p, uint8_t* base, Sm* sm, uint32_t tmem, int warp, int lane) {
  const int w = warp & 3, row = 32 * w + lane;
  const uint32_t ts = tmem + ((uint32_t)(32 * w) << 16) + kTmS;
  uint8_t* sb = base + kOffS;
  bool failed = false;
  Rec r{};
  int ci = 0, ins = 0, fins = 0, outs = 0;  // chunks; 16-bit and f32 states by TMA that came, states that went
  int entries = 0;                          // of the stages of K and V
  auto load_in = [&](int c0, uint32_t (&x)[32]) {
    if (kWide && r.in >= 0) {
      load_state32<kWide>(p.ws, kF32, (int64_t)r.in * (D * D) + row * D + c0, x);
    } else if (r.in == kPool && p.s_in) {
      load_state32<kWide>(p.s_in, p.sin_dtype, (int64_t)r.slot * p.sin_slot + (int64_t)r.h * p.sin_head + row * D + c0, x);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = 0u;
    }
  };
  auto store_out = [&](int c0, const uint32_t (&x)[32]) {
    const int64_t at = row * D + c0;
    if (kWide && r.out >= 0) store_state32<kWide>(p.ws, kF32, (int64_t)r.out * (D * D) + at, x);
    else store_state32<kWide>(p.s_out, p.sout_dtype, (int64_t)r.slot * p.sout_slot + (int64_t)r.h * p.sout_head + at, x);
  };
  // S <- b S + (a S + what the chunk before added, from TMEM); with `copy`, also in 16 bits to where Q S^T reads it
  float2 S[apart<kWide>() ? D / 2 : 1];
  float sa = 0.f, keep = 0.f;  // a and b
  auto put_copy = [&](int q) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<uint4*>(sb + (q >> 1) * kHalf + sw128_chunk(row, 4 * (q & 1) + e)) =
          make_uint4(pack16x2<F16>(S[16 * q + 4 * e]), pack16x2<F16>(S[16 * q + 4 * e + 1]),
                     pack16x2<F16>(S[16 * q + 4 * e + 2]), pack16x2<F16>(S[16 * q + 4 * e + 3]));
  };
  auto add_chunk = [&](uint32_t from, int v_exp, bool copy) {
    const float2 a2 = pair(sa), b2 = pair(keep), f2 = pair(__int_as_float((127 - v_exp) << 23));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t x[32];
      tmem_ld32(from + 32 * q, x);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; ++e)
        S[16 * q + e] = fma2(b2, S[16 * q + e], fma2(a2, S[16 * q + e], lifted<F16, kWide>() ? mul2(f2, pair_at(x + 2 * e)) : pair_at(x + 2 * e)));
      if (copy) put_copy(q);
    }
  };
  auto v_exp = [&](int chunk) { return lifted<F16, kWide>() ? (int)sm->v_exp[chunk & 3][2 * w + (lane >> 4)] : 0; };
  auto zero = [&] {
#pragma unroll
    for (int e = 0; e < D / 2; ++e) S[e] = make_float2(0.f, 0.f);
  };
  auto put_back = [&](uint32_t to) {  // S to TMEM, from where loops that are rolled up store it
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) { x[2 * e] = __float_as_uint(S[4 * q + e].x); x[2 * e + 1] = __float_as_uint(S[4 * q + e].y); }
      tmem_st8(to + 8 * q, x);
    }
    tmem_st_wait();
  };
  for (int u = 0; next_unit(sm, u, lane, &r, &failed); ++u) {
    const bool ring = !kStates && state_in_ring<kWide>(p, r);
    const uint8_t* from = base + kOffKv + (entries & 1) * 2 * kTile;
    entries += r.nch + ring;
    for (int c = 0; c < r.nch && kStates; ++c, ++ci) {
      if (!wait(sm, &sm->sum_done[ci & 1], (ci >> 1) & 1)) { failed = true; break; }
      tc_fence_after();
      if (c == 0) zero();
      keep = 1.f;
      add_chunk(ts + (sum_col<kStates>(ci) - kTmS), v_exp(ci), false);
      if (c + 1 == r.nch) continue;
      tc_fence_before();
      warp_arrive(&sm->sum_free[ci & 1], lane);
    }
    for (int c = 0; c < r.nch && !kStates; ++c, ++ci) {
      const int st = ci & 1;
      // S as the chunk finds it: to 16 bits for Q S^T, times the chunk's decay for V_d^T K
      if (!(wait(sm, &sm->gate_full[st], (ci >> 1) & 1) && (c == 0 || wait(sm, &sm->s_done, (ci - 1) & 1)))) { failed = true; break; }
      tc_fence_after();
      const float2 gam = pair(sm->gamma[st]);
      const bool direct = c == 0 && state_in_tma<kWide>(p, r);  // the copy came by TMA
      if (c == 0 && !(direct ? wait(sm, &sm->si_full, ins++ & 1) : outs == 0 || wait(sm, &sm->f_stored, (outs - 1) & 1))) {
        failed = true;
        break;
      }
      if (c == 0 && ring && !wait(sm, &sm->sf_full, fins++ & 1)) { failed = true; break; }
      auto through = [&] {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t x[32];
          if (c > 0) {
            tmem_ld32(ts + 32 * q, x);
            tmem_ld_wait();
          } else if (direct) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 z = *reinterpret_cast<const uint4*>(sb + (q >> 1) * kHalf + sw128_chunk(row, 4 * (q & 1) + e));
              const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = unpack16<F16>(zw[i]);
                x[8 * e + 2 * i] = __float_as_uint(f.x);
                x[8 * e + 2 * i + 1] = __float_as_uint(f.y);
              }
            }
          } else {
            load_in(32 * q, x);
          }
          if (!apart<kWide>()) {
#pragma unroll
            for (int e = 0; e < 4 && !direct; ++e)
              *reinterpret_cast<uint4*>(sb + (q >> 1) * kHalf + sw128_chunk(row, 4 * (q & 1) + e)) =
                  make_uint4(pack16x2<F16>(pair_at(x + 8 * e)), pack16x2<F16>(pair_at(x + 8 * e + 2)),
                             pack16x2<F16>(pair_at(x + 8 * e + 4)), pack16x2<F16>(pair_at(x + 8 * e + 6)));
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = mul2(pair_at(x + e), gam);
              x[e] = __float_as_uint(y.x);
              x[e + 1] = __float_as_uint(y.y);
            }
          }
          tmem_st32(ts + 32 * q, x);
        }
      };
      if (!apart<kWide>()) {
        through();
      } else {
        if (c == 0 && ring) {  // an f32 state out of a stage of K and V
#pragma unroll
          for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 z = *reinterpret_cast<const float4*>(from + q * kHalf + sw128_chunk(row, e));
              S[16 * q + 2 * e] = make_float2(z.x, z.y);
              S[16 * q + 2 * e + 1] = make_float2(z.z, z.w);
            }
            put_copy(q);
          }
        } else {
          if (c == 0) {  // another, or none, to TMEM as it is: it is what is added to zero
            through();
            tmem_st_wait();
            zero();
          }
          add_chunk(ts, c == 0 ? 0 : v_exp(ci - 1), !direct);
        }
        sa = sm->gamma[st];
        keep = __float_as_int(sa) < 0 ? 1.f : 0.f;
      }
      fence_proxy_async_smem();
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&sm->s_ready, lane);
      if (lane == 0) mbar_arrive(&sm->gate_empty[st]);
      if (c == 0 && ring && lane == 0) mbar_arrive(&sm->sf_empty);
    }
    if (failed) break;
    // the state that the unit leaves; the next unit may overwrite TMEM and the 16-bit copy after
    // that, Q S^T having run before
    if (!kStates && !wait(sm, &sm->s_done, (ci - 1) & 1)) { failed = true; break; }
    if (r.out == kNone || (r.out == kPool && !p.s_out)) continue;
    tc_fence_after();
    const uint32_t last = ts + (sum_col<kStates>(ci - 1) - kTmS);
    if (apart<kWide>()) {
      if (!kStates) add_chunk(last, v_exp(ci - 1), false);
      put_back(last);
    }
    if (!kStates && kWide && state_out_tma(p, r) && p.sout_dtype == kF32) {
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t x[32];
        tmem_ld32(ts + 32 * q, x);
        tmem_ld_wait();
        if (q == 2 && !wait(sm, &sm->f_half, outs & 1)) { failed = true; break; }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(sb + (q & 1) * kHalf + sw128_chunk(row, e)) =
              make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        if (q & 1) {
          fence_proxy_async_smem();
          warp_arrive(&sm->f_staged, lane);
        }
      }
      if (failed) break;
      ++outs;
      continue;
    }
    if (!kStates && state_out_tma(p, r)) {
      ++outs;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t x[32];
        tmem_ld32(ts + 32 * q, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = pair_at(x + 8 * e + 2 * i);
            y[i] = p.sout_dtype == kF16 ? pack16x2<true>(f) : pack16x2<false>(f);
          }
          *reinterpret_cast<uint4*>(sb + (q >> 1) * kHalf + sw128_chunk(row, 4 * (q & 1) + e)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      fence_proxy_async_smem();
      warp_arrive(&sm->f_staged, lane);
      continue;
    }
    const bool start = kStates && r.in == kPool && p.s_in;
    const float2 whole = pair(start ? p.ws_decay[r.out] : 0.f);
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      uint32_t x[32];
      tmem_ld32(last + 32 * q, x);
      tmem_ld_wait();
      if (start) {  // what the segment added, and the state that it started from
        uint32_t y[32];
        load_in(32 * q, y);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 z = fma2(pair_at(y + e), whole, pair_at(x + e));
          x[e] = __float_as_uint(z.x);
          x[e + 1] = __float_as_uint(z.y);
        }
      }
      store_out(32 * q, x);
    }
    if (kStates) {
      tc_fence_before();
      warp_arrive(&sm->sum_free[(ci - 1) & 1], lane);
    }
  }
  if (failed) {
    if (lane == 0) give_up(p, sm);
    return;
  }
  // units without chunks pass on what they got: 32 units looked at together, a lane each
  const int64_t units = r.h > 0 ? unit_count<kStates>(p) : 0;
  for (int64_t x0 = blockIdx.x; x0 < units; x0 += 32 * (int64_t)gridDim.x) {
    const int64_t x = x0 + (int64_t)lane * gridDim.x;
    Rec mine{};
    bool empty = x < units && unit_at<kStates>(p, x, &mine) == 0 && mine.nch == 0;
    for (unsigned left = __ballot_sync(0xffffffffu, empty); left; left &= left - 1) {
      const int from = __ffs(left) - 1;
      r.h = __shfl_sync(0xffffffffu, mine.h, from);
      r.in = __shfl_sync(0xffffffffu, mine.in, from);
      r.out = __shfl_sync(0xffffffffu, mine.out, from);
      r.slot = __shfl_sync(0xffffffffu, mine.slot, from);
      if (kStates && w == 0 && lane == 0) p.ws_decay[r.out] = 1.f;
      if (r.out == kNone || (r.out == kPool && !p.s_out)) continue;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t y[32];
        load_in(32 * q, y);
        store_out(32 * q, y);
      }
    }
  }
}

// ------------------------------------------------------------ warps 16-23: V_d
// Transposed fragments of V (pairs of tokens, one value each) times d, as kTerms 16-bit terms, 16
// values a warp.  Where only states are made, the warps of P do the same, every other part.
template <bool F16, int kTerms, bool kStates, bool kWide, class Sm>
__device__ __forceinline__ void run_v(const DecayPrefillParams& p, uint8_t* base, Sm* sm, uint32_t tmem, int warp, int lane) {
  constexpr int kSub = sub_tokens<kTerms>(), kSubs = C / kSub, kGroups = kStates ? 2 : 1;
  constexpr bool kLifted = lifted<F16, kWide>();
  const int w = warp & 3, hf = (warp >> 2) & 1, group = kStates && warp < 4 + kPoWarps ? 1 : 0;
  const uint32_t tq = tmem + ((uint32_t)(32 * w + 16 * hf) << 16);
  const int m = lane >> 3, lr = lane & 7;
  const int ch = 4 * w + 2 * hf + (m & 1);  // this lane's 16-byte chunk of a row of V
  bool failed = false;
  Rec r;
  int ci = 0;
  Ring<kStates> ring;
  for (int u = 0; next_unit(sm, u, lane, &r, &failed); ++u) {
    if (!kStates && state_in_ring<kWide>(p, r)) ring.pass();
    for (int c = 0; c < r.nch; ++c, ++ci, ring.next()) {
      const int st = ci & 1, left = r.len - (kStates ? r.nch - 1 - c : c) * C;
      const int kv = ring.s;
      const uint32_t ph = ring.phase();
      if (!(wait(sm, &sm->gate_full[st], (ci >> 1) & 1) && wait(sm, &sm->v_full[kv], ph))) { failed = true; break; }
      uint8_t* k = base + kOffKv + kv * 2 * kTile;
      if (left < C) {
        if (!wait(sm, &sm->k_full[kv], ph)) { failed = true; break; }
        zero_tails<kSub, kLifted ? 1 : kGroups>(k, k + kTile, left, 4 * w + 2 * hf, kLifted ? 0 : group, lane);
      }
      const uint32_t va = smem_u32(k + kTile) + (ch >> 3) * kHalf;
      const int up = kLifted ? v_scale(va, m, lr, ch) : 0;
      const __half2 scale = __half2half2(__ushort_as_half((unsigned short)((up + 15) << 10)));
      auto scaled = [&](uint32_t x) {
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x), scale);
        return *reinterpret_cast<const uint32_t*>(&y);
      };
#pragma unroll 1
      for (int sub = group; sub < kSubs; sub += kGroups) {
        int slot, round;
        vd_place<kTerms, kStates>(ci, sub, &slot, &round);
        if (!((round == 0 || wait(sm, &sm->vd_empty[slot], (round - 1) & 1)) &&
              (kStates || slot != 1 || wait(sm, &sm->qs_done, ci & 1)) &&
              (kStates || slot != 2 || wait(sm, &sm->cf_empty, ci & 1)))) { failed = true; break; }
        tc_fence_after();
        // behind a wait for a product that added this chunk's predecessor, so that what was here has been read
        if (kLifted && sub == 0 && lane == 0) sm->v_exp[ci & 3][2 * w + hf] = (int8_t)(up + kDExp);
#pragma unroll 2
        for (int tt = 0; tt < kSub / 16; ++tt) {
          const int tok = sub * kSub + 16 * tt;  // 16 tokens from here
          const int at2 = (tok >> 1) + (lane & 3);  // this lane's first pair of tokens; the second is 4 pairs on
          const uint32_t to = tq + vd_slot_col<kStates>(slot) + 8 * tt;
          uint32_t a[4], t[4];
          ldmatrix_x4_trans(va + sw128_chunk(tok + (m >> 1) * 8 + lr, ch & 7), a);
          if (kTerms == 2) {
            // three packed 16-bit operations
            const uint32_t* dh = reinterpret_cast<const uint32_t*>(sm->d[st]) + at2;
            uint32_t rest[4], h[2] = {dh[0], dh[4]}, l[2] = {dh[C / 2], dh[C / 2 + 4]};
            if (kLifted) {
              if (up > 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = scaled(a[e]);
              } else if (up < 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) { h[e] = scaled(h[e]); l[e] = scaled(l[e]); }
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) split_product<F16>(a[e], h[e >> 1], l[e >> 1], &t[e], &rest[e]);
            tmem_st16x128_x2(to, t);
            tmem_st16x128_x2(to + kSub / 2, rest);
          } else {
            float2 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = mul2(unpack16<F16>(a[e]), reinterpret_cast<const float2*>(sm->d[st])[at2 + 2 * (e & 2)]);
#pragma unroll
            for (int term = 0; term < kTerms; ++term) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                t[e] = pack16x2<F16>(x[e]);
                if (term + 1 < kTerms) x[e] = fma2(unpack16<F16>(t[e]), pair(-1.f), x[e]);
              }
              tmem_st16x128_x2(to + term * (kSub / 2), t);
            }
          }
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm->vd_full[slot], lane);
      }
      if (failed) break;
      if (lane == 0) mbar_arrive(&sm->gate_empty[st]);
    }
    if (failed) break;
  }
  if (failed && lane == 0) give_up(p, sm);
}

// ------------------------------------------------------------ the kernel
template <bool F16, int kTerms, bool kStates, bool kWide, bool kClaim>
__global__ void __launch_bounds__(kThreads, 1) gdn_decay_prefill_kernel(const __grid_constant__ DecayPrefillParams p) {
  extern __shared__ __align__(1024) uint8_t base[];
  using Sm = Small<kStates, apart<kWide>()>;
  Sm* sm = reinterpret_cast<Sm*>(base + kOffSmall);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    auto init = [](uint64_t* bar, int n, int count) {
      for (int i = 0; i < n; ++i) mbar_init(bar + i, count);
    };
    init(&sm->q_full, 1, 1);
    init(&sm->q_empty, 1, kPoWarps);
    init(sm->k_full, kv_stages<kStates>(), 1);
    init(sm->v_full, kv_stages<kStates>(), 1);
    init(sm->kv_empty, kv_stages<kStates>(), 1);
    init(sm->rec_full, kRecs, 1);
    init(sm->rec_empty, kRecs, (kStates ? 2 : 3) + kPoWarps + kSWarps + kVWarps);
    init(sm->gate_full, 2, p.hold_gates ? 2 : 1);  // held: one arrival of two never comes
    init(sm->gate_empty, 2, kPoWarps + (kStates ? 0 : kSWarps) + kVWarps);
    init(&sm->claim_full, 1, 1);
    init(&sm->cf_empty, 1, kPoWarps);
    if (kStates) {
      init(sm->sum_done, 2, 1);
      init(sm->sum_free, 2, kSWarps);
    } else {
      init(&sm->qk_done, 1, 1);
      init(&sm->qs_done, 1, 1);
      init(&sm->s_done, 1, 1);
      init(&sm->o_done, 1, 1);
    }
    init(&sm->p_ready, 1, kPoWarps);
    init(&sm->o_free, 1, kPoWarps);
    init(&sm->o_staged, 1, kPoWarps);
    init(&sm->q_ready, 1, kPoWarps);
    init(&sm->o_stored, 1, 1);
    init(&sm->f_half, 1, 1);
    init(&sm->f_stored, 1, 1);
    init(&sm->f_staged, 1, kSWarps);
    init(&sm->si_full, 1, 1);
    init(&sm->sf_full, 1, 1);
    init(&sm->sf_empty, 1, kSWarps);
    init(&sm->s_ready, 1, kSWarps);
    init(sm->vd_full, vd_slots<kStates>(), kVWarps);
    init(sm->vd_empty, vd_slots<kStates>(), 1);
    init(&sm->drain, 1, 1);
    sm->abort = 0;
    sm->tries = (int32_t)max(uint64_t(1), min(p.wait_ns ? p.wait_ns : kWaitNs, kWaitNs) / (Sm::kInline ? kProbeInlineNs : kProbeNs));
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
    tma_prefetch_desc(&p.tm_o);
  }
  if (warp == 0) {
    tmem_alloc(&sm->tmem, kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;
  if (warp < 4) {
    if (apart<kWide>()) reg_dec<kRegsOne>();
    if (warp == 0) run_producer<kStates, kWide, kClaim>(p, base, sm, lane);
    else if (warp == 1) run_mma<F16, kTerms, kStates, kWide>(p, base, sm, tmem, lane);
    else if (warp == 2) run_gates<F16, kTerms, kStates, kWide>(p, sm, lane);
    else if (!kStates) run_store<kWide>(p, base, sm, lane);
  } else if (warp < 4 + kPoWarps) {
    if (apart<kWide>()) reg_dec<kRegsPo>();
    if (kStates) run_v<F16, kTerms, kStates, kWide>(p, base, sm, tmem, warp, lane);
    else run_po<F16, kWide>(p, base, sm, tmem, warp, lane);
  } else if (warp < 4 + kPoWarps + kSWarps) {
    if (apart<kWide>()) reg_inc<kRegsState>();
    run_state<F16, kTerms, kStates, kWide>(p, base, sm, tmem, warp, lane);
  } else {
    if (apart<kWide>()) reg_dec<kRegsV>();
    run_v<F16, kTerms, kStates, kWide>(p, base, sm, tmem, warp, lane);
  }
  tmem_st_wait();  // of a role that has given up
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmCols);
}

// ------------------------------------------------------------ joining segments
// In f32, the state behind each segment: S <- decay S + what the segment added.  A thread takes
// four values of one unit through all segments, and loads those of the next few segments while it
// works on the last few.
constexpr int kJoinThreads = 256, kJoinAhead = 8;
__global__ void __launch_bounds__(kJoinThreads) gdn_decay_join_kernel(float* __restrict__ ws, const float* __restrict__ decay, int blocks) {
  constexpr int kCtas = D * D / 4 / kJoinThreads;  // of a unit
  const int64_t unit = blockIdx.x / kCtas;
  float4* s = reinterpret_cast<float4*>(ws + unit * blocks * (D * D)) + (blockIdx.x % kCtas) * kJoinThreads + threadIdx.x;
  const float* d = decay + unit * blocks;
  float4 next[kJoinAhead];
  float g_next[kJoinAhead];
  auto load = [&](int b0) {
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) {
      next[i] = b0 + i < blocks ? s[(b0 + i) * (D * D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
      g_next[i] = b0 + i < blocks ? d[b0 + i] : 0.f;
    }
  };
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  load(0);
  for (int b0 = 0; b0 < blocks; b0 += kJoinAhead) {
    float4 y[kJoinAhead];
    float g[kJoinAhead];
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) { y[i] = next[i]; g[i] = g_next[i]; }
    load(b0 + kJoinAhead);
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) {
      if (b0 + i == 0) {
        x = y[0];  // already what is behind the first segment
      } else if (b0 + i < blocks) {
        x = make_float4(fmaf(g[i], x.x, y[i].x), fmaf(g[i], x.y, y[i].y), fmaf(g[i], x.z, y[i].z), fmaf(g[i], x.w, y[i].w));
        s[(b0 + i) * (D * D / 4)] = x;
      }
    }
  }
}

// Whether CTAs take units over instead of walking them in equal steps.  That evens out sequences of
// different lengths, but each claim delays what follows by about a microsecond: it pays where an SM
// has few units, or long ones.  Us in equal steps and by claims, lengths drawn evenly up to twice the mean: 93
// sequences of 1198 tokens on 2 heads 113 / 78, 64 x 2000 on 16 348 / 313, 300 x 1000 on 16 870 / 806, 400 x 600
// on 8 347 / 348, 200 x 136 on 16 137 / 145, 1000 x 300 on 16 948 / 1042.
bool claims_pay(int64_t units, double chunks, int sms) {
  return units > sms && chunks >= (units <= 8 * (int64_t)sms ? 2.0 : 6.0);
}

template <bool F16, int kTerms, bool kStates, bool kWide, bool kClaim>
cudaError_t launch_walk(const DecayPrefillParams& p, int sms, cudaStream_t stream) {
  static thread_local int device = -1, generation = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const int gen = launch_config_generation();
  if (e == cudaSuccess && (device != dev || generation != gen)) {
    e = cudaFuncSetAttribute(gdn_decay_prefill_kernel<F16, kTerms, kStates, kWide, kClaim>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    cudaFuncAttributes have{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&have, gdn_decay_prefill_kernel<F16, kTerms, kStates, kWide, kClaim>);
    // the shares of the groups of warps are those of kRegs: with fewer, the group that asks for more would wait for ever
    if (e == cudaSuccess && apart<kWide>() && have.numRegs <= kRegs - 8) e = cudaErrorLaunchOutOfResources;
    if (e == cudaSuccess) { device = dev; generation = gen; }
  }
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.N * p.H * (kStates ? p.splits - 1 : p.splits);
  const int64_t grid = kClaim || units < sms ? units : sms;
  gdn_decay_prefill_kernel<F16, kTerms, kStates, kWide, kClaim><<<(unsigned)grid, kThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <bool F16, int kTerms, bool kStates, bool kWide>
cudaError_t launch_pass(const DecayPrefillParams& p, int sms, cudaStream_t stream) {
  const int64_t units = (int64_t)p.N * p.H * (kStates ? p.splits - 1 : p.splits);
  return claims_pay(units, double(p.T) / double(p.N) / p.splits / C, sms)
             ? launch_walk<F16, kTerms, kStates, kWide, true>(p, sms, stream)
             : launch_walk<F16, kTerms, kStates, kWide, false>(p, sms, stream);
}

template <bool F16, int kTerms>
cudaError_t launch(const DecayPrefillParams& p, cudaStream_t stream) {
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (p.splits > 1) {
    cudaError_t e = launch_pass<F16, kTerms, true, true>(p, sms, stream);
    if (e != cudaSuccess) return e;
    if (p.splits > 2) {
      const int64_t ctas = (int64_t)p.N * p.H * (D * D / 4 / kJoinThreads);
      gdn_decay_join_kernel<<<(unsigned)ctas, kJoinThreads, 0, stream>>>(p.ws, p.ws_decay, p.splits - 1);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  }
  if constexpr (kTerms == 2) {  // three terms are for a state that stays in f32, whether it is asked for or not
    // f16 inputs: a bf16 state takes the way of f32 ones, as it holds more of small values than f16 does
    const bool wide = p.splits > 1 || (p.s_in && p.sin_dtype == kF32) || (p.s_out && (p.sout_dtype == kF32 || (F16 && p.sout_dtype == kBF16)));
    if (!wide) return launch_pass<F16, kTerms, false, false>(p, sms, stream);
  }
  return launch_pass<F16, kTerms, false, true>(p, sms, stream);
}

}  // namespace

// Time in chunks of the main pass, with U units on a persistent grid of one CTA an SM: rounds times
// the chunks of a unit and what a unit costs besides.  Cut into P segments, U P units go through the
// main pass and U (P - 1) through the pass that makes states (no scores, no output, two of four
// products), and the join walks P - 1 states.  A cut has to save a twentieth, and leaves two chunks
// or more to a segment.  The constants are a fit to measured times of 12 shapes from 4 x 2000 to
// 32 x 131072 (heads x tokens of a sequence), each uncut and in 2 to 152 segments; the P that it
// picks is the fastest one measured in each (32000 tokens on 8 heads: 575 us uncut, 78 in 18
// segments, 114 in 22; 2 x 65536 on 32 heads: 1457 uncut, 990 in 7, 1250 in 3; 16 x 4096 on 32: 316
// uncut, 400 in 2).
int decay_splits(int64_t units, double chunks, int sms) {
  constexpr double kUnit = 2.5, kStatesChunk = 0.35, kStatesUnit = 0.75, kLaunches = 3.0, kJoin = 0.06;
  if (units <= 0 || sms <= 0) return 1;
  auto rounds = [&](int64_t n) { return double((n + sms - 1) / sms); };
  double best = 0.95 * rounds(units) * (std::ceil(chunks) + kUnit);
  int P = 1;
  for (int c = 2; c <= sms && chunks >= 2.0 * c; ++c) {
    const double each = std::ceil(chunks / c);
    const double cost = rounds(units * c) * (each + kUnit) + rounds(units * (c - 1)) * (kStatesChunk * each + kStatesUnit) +
                        kLaunches + kJoin * (c - 1);
    if (cost < best) { best = cost; P = c; }
  }
  return P;
}

cudaError_t launch_decay_prefill(const DecayPrefillParams& p, cudaStream_t stream) {
  if ((int64_t)p.N * p.H <= 0) return cudaSuccess;
  if (p.op_f16) return launch<true, 2>(p, stream);
  if (p.s_out && p.sout_dtype != kF32) return launch<false, 2>(p, stream);
  return launch<false, 3>(p, stream);
}

}  // namespace gdn
