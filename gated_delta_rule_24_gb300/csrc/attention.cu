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
// The prefix has units of its own: with up to 16 rows a key head in all, they are walked behind the sequences' ones; with more,
// 256 rows a unit go to the tensor cores (attention_prefix.cuh), which they keep busy while the own pages (attention_own.cuh) keep
// HBM busy: one kernel then shares the SMs out between the two kinds of workers, as the lengths on the
// device ask for.
//
// Measured as one call in a graph: 511 keys of one sequence 8.4 us, which is two kernels' start and the way of one tile; the rest
// stands with the two kinds of workers.
#include "attention_own.cuh"
#include "attention_prefix.cuh"

#include <algorithm>

namespace gdn {
namespace {

constexpr int kResident = 2;  // workers of the own pages on an SM

// Whether the swizzled tiles would not be where they have to be; there is no room to spare for it.  It is so for all CTAs then: none has a
// share, and no unit has a worker, so that the join does not take the workspace's for an earlier call's.
__device__ __forceinline__ bool misplaced(const AttentionParams& p, const uint8_t* smem) {
  if (!(smem_u32(smem) & 1023)) return false;
  if (threadIdx.x == 0) atomicOr(p.dev_err, kDevErrTimeout);
  const int64_t places = 2 * ((p.last_worker - p.first_worker) + (p.prefix_last - p.prefix_first));   // one array
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < places; i += (int64_t)gridDim.x * blockDim.x) p.first_worker[i] = -1;
  return true;
}

// One worker of the own pages (and of a prefix of few rows) a CTA.
template <bool F16, int kEights>
__global__ void __launch_bounds__(own::kThreads, kResident) gdn_attention_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  grid_wait();
  if (misplaced(p, smem)) return;
  go_ahead();
  if (threadIdx.x == 0 && p.pages > 0) {
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  own::Count count;
  count.make(p, own::bars_of(smem), reinterpret_cast<uint32_t*>(smem), threadIdx.x, 1);
  // no more shares than there is to share: one without anything between two parts of a unit would leave a gap
  const uint32_t shares = min(own::whole_cost(p, count), gridDim.x / p.blocks_aside);
  if (blockIdx.x >= shares * p.blocks_aside) return;
  own::run_worker<F16, kEights, false>(p, smem, threadIdx.x, count, blockIdx.x, shares, 1);
}

// SMs out of `sms` for the own pages beside a prefix of many rows, by what the two take an SM: 0.34 us for a tile's cost of 16 rows (two
// workers side by side), 0.32 of 8, 1.4 us for 128 keys of 256 rows.  us with 0.25, 0.29, 0.32, 0.34, 0.37 and 0.42:
//   256 sequences of 8 rows a key head and 512 keys behind 32768    129 134 123 125 125 132
//   100 of 7 rows, 300 keys, behind 20000                           42 41 40 40 40 42
//   300 of 8 rows, 100 keys, one key head, behind 50000             60 58 55 55 56 57
//   200 of 2 rows, 1000 keys, 8 key heads, behind 10000             148 147 150 151 151 154
//   64 of 16 rows, 1500 keys, behind 30000                          87 80 76 76 71 71
// A prefix of up to 128 rows is held by HBM, too, and loses little by an SM less, while the own pages get on more slowly beside it: 0.9 there.
// us with 0.34, 0.5, 0.7, 0.9, 1.2 and 1.6:
//   64 rows, 300 own keys, behind 100000     48 46 46 46 46 46       64 rows, 3000 own keys     54 51 52 52 53 54
//   128 rows, 500, behind 65536              45 43 43 43 43 43       128 rows on two key heads  28 24 23 23 23 23
//   160 rows, 500, behind 65536              45 45 45 45 46 46       256 rows                   48 49 49 49 51 53
//   512 rows, 500, behind 32768              42 46 48 50 55 62
template <int kEights>
__device__ __forceinline__ int sms_for_own(uint32_t own_cost, int aside, uint32_t prefix_cost, bool few_rows, int sms) {
  if (own_cost == 0) return 0;
  const float own = (few_rows ? 0.9f : kEights == 1 ? 0.32f : 0.34f) * own_cost * aside, prefix = 1.4f * prefix_cost;
  return max((aside + 1) / 2, min((int)(sms * (own / (own + prefix)) + 0.5f), sms - 1));
}

// The own pages and a prefix of many rows side by side: a CTA is one worker of the prefix, or two of the own pages.
template <bool F16, int kEights>
__global__ void __launch_bounds__(prefix::kThreads, 1) gdn_attention_both_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  grid_wait();
  if (misplaced(p, smem)) return;
  go_ahead();
  if (threadIdx.x == 0 && p.pages > 0) {
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
    tma_prefetch_desc(&p.tm_pk);
    tma_prefetch_desc(&p.tm_pv);
  }
  // two groups of threads count the tiles, each for a worker that it may be, and tell the rest
  uint32_t* room = reinterpret_cast<uint32_t*>(smem);
  const int half = threadIdx.x / own::kThreads, tid = threadIdx.x - half * own::kThreads;
  own::Count count;
  if (half < 2) count.make(p, own::bars_of(smem + half * own::kPlace), room + 8 * half, tid, 1 + half);
  if (threadIdx.x == 0) { room[16] = count.all.tiles; room[17] = count.all.cost; }
  __syncthreads();
  count.all = {room[16], room[17]};
  fence_proxy_async_smem();
  __syncthreads();
  const uint32_t tiles = (p.prefix + kPrefixKeys - 1) / kPrefixKeys, steps = p.H_k * p.prefix_units * (tiles + prefix::kUnitCost);
  const uint32_t own_cost = own::whole_cost(p, count);
  const int own_sms = sms_for_own<kEights>(own_cost, p.blocks_aside, steps, p.N * p.tokens * p.group <= kPrefixRows / 2, gridDim.x), prefix_workers = min(steps, gridDim.x - own_sms);
  if (blockIdx.x < prefix_workers) {
    prefix::run_worker<F16>(p, smem, blockIdx.x, prefix_workers);
  } else if (blockIdx.x >= gridDim.x - own_sms) {
    const uint32_t worker = 2 * (blockIdx.x - (gridDim.x - own_sms)) + half, shares = min(own_cost, (uint32_t)(2 * own_sms / p.blocks_aside));
    if (half < 2 && worker < shares * p.blocks_aside)
      own::run_worker<F16, kEights, true>(p, smem + half * own::kPlace, tid, count, worker, shares, 1 + half);
  }
}

// The parts of the units that were cut, and those of the prefix: `kPer` warps for each row take turns at its
// parts, kBatch on their way at a time, lanes four columns each.
template <int kPer> constexpr int kJoinThreads = 32 * (kPer > 4 ? kPer : 4);
template <bool F16, int kPer, int kBatch>
__global__ void __launch_bounds__(kJoinThreads<kPer>) gdn_attention_join_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int kRowsHere = kJoinThreads<kPer> / 32 / kPer;
  __shared__ float s_o[kPer][kHeadDim];
  __shared__ float2 s_ml[kPer];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5 & (kPer - 1);
  const uint32_t id = blockIdx.x * kRowsHere + threadIdx.x / (32 * kPer), subs = p.H_k * p.blocks;
  const uint32_t unit = over(id, p.by_rows), row = id - unit * p.block_rows, n = over(unit, p.by_subs), sub = unit - n * subs, hk = over(sub, p.by_blocks);
  const int r = (sub - hk * p.blocks) * own::kRows + row;
  const bool some = n < (uint32_t)p.N && r < p.tokens * p.group;
  // the row of the prefix, and its unit of the prefix kernel's or of the walk's
  const uint32_t pr = n * p.tokens * p.group + r;
  const bool many = p.prefix_units > 0;
  const uint32_t prefix_unit = many ? hk * p.prefix_units + pr / kPrefixRows : p.N * subs + hk * p.prefix_blocks + pr / own::kRows;
  grid_wait();
  // The length, and the sequence's own parts: of the workers from the first to the last (one side of the shares), or one of a whole unit;
  // then the prefix'.  All are asked for at once, and where there are no keys an earlier call's are not looked at.
  int length = -1, first = 0, last = 0, prefix_first = 0, prefix_last = -1;
  if (some) {
    length = length_of(p, n);
    first = p.first_worker[unit];
    last = p.last_worker[unit];
    if (p.prefix) {
      prefix_first = (many ? p.prefix_first : p.first_worker)[prefix_unit];
      prefix_last = (many ? p.prefix_last : p.last_worker)[prefix_unit];
    }
  }
  if (length < 0) {  // reported here, as there may be nothing for the kernel before this one to do, and it is not launched then
    if (some && sub == 0 && row == 0 && (threadIdx.x & (32 * kPer - 1)) == 0) atomicOr(p.dev_err, kDevErrLength);
    return;
  }
  // parts of no worker: the kernel before this one gave up, and said so
  bool bad = (length > 0 && (first < 0 || last < first || last >= p.workers)) ||
             (p.prefix && (prefix_first < 0 || prefix_last < prefix_first || prefix_last >= (many ? p.prefix_workers : p.workers)));
  int own = length > 0 && !bad ? over(last - first, p.by_aside) + 1 : 0, shared = bad ? 0 : prefix_last - prefix_first + 1;
  if (own == 1 && !p.prefix) return;  // it is in the output
  float top = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < own + shared; i0 += kBatch * kPer) {
    float2 ml[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = i0 + e * kPer;
      ml[e] = make_float2(-INFINITY, 0.f);
      x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i >= own + shared) continue;
      if (i >= own && many) {
        const int w = prefix_first + i - own;
        const int64_t slot = shared == 1 ? 2 * (int64_t)p.prefix_workers + prefix_unit : 2 * w + (i == own ? 1 : 0);
        ml[e] = *reinterpret_cast<const float2*>(p.prefix_ml + 2 * (slot * kPrefixRows + pr % kPrefixRows));
        x[e] = *reinterpret_cast<const float4*>(p.prefix_o + (slot * kHeadDim + lane / 2 * 8) * kPrefixRows + pr % kPrefixRows * 8 + (lane & 1) * 4);
      } else {
        const bool of_prefix = i >= own;
        const int w = of_prefix ? prefix_first + i - own : first + i * p.blocks_aside;
        const int64_t slot = (of_prefix ? shared : own) == 1 ? 2 * (int64_t)p.workers + (of_prefix ? prefix_unit : unit) : 2 * w + (i == 0 || i == own ? 1 : 0);
        const int64_t at = slot * p.block_rows + (of_prefix ? pr % own::kRows : row);
        ml[e] = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
        x[e] = *reinterpret_cast<const float4*>(p.part_o + at * kHeadDim + 4 * lane);
      }
    }
    float now = top;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      now = fmaxf(now, ml[e].x);
      bad |= ml[e].y == kAttentionBad;
    }
    const float from_base = now == -INFINITY ? 0.f : now, keep = exp2_fast(top - from_base);
    top = now;
    l *= keep;
    o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
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
    const float2 ml = lane < kPer ? s_ml[lane] : make_float2(-INFINITY, 0.f);
    top = ml.x;
#pragma unroll
    for (int d = kPer / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float f = exp2_fast(ml.x - (top == -INFINITY ? 0.f : top));
    l = f * ml.y;
#pragma unroll
    for (int d = kPer / 2; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int w = 0; w < kPer; ++w) {
      const float fw = __shfl_sync(0xffffffffu, f, w);
      const float4 x = reinterpret_cast<const float4*>(s_o[w])[lane];
      o = make_float4(fmaf(fw, x.x, o.x), fmaf(fw, x.y, o.y), fmaf(fw, x.z, o.z), fmaf(fw, x.w, o.w));
    }
    top = __shfl_sync(0xffffffffu, top, 0);
    l = __shfl_sync(0xffffffffu, l, 0);
  }
  if (bad) return;
  const float from_base = top == -INFINITY ? 0.f : top;
  const bool none = top == -INFINITY && l == 0.f;
  const float inv = none ? 0.f : inverse(l);
  const int of_unit = over(r, p.by_group), head = hk * p.group + r - of_unit * p.group;
  const int64_t token = n * (int64_t)p.tokens + of_unit;
  *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + token * p.o_st + head * p.o_sh + 4 * lane) =
      make_uint2(pack16x2<F16>(o.x * inv, o.y * inv), pack16x2<F16>(o.z * inv, o.w * inv));
  if (p.lse && lane == 0) p.lse[token * p.lse_st + head] = none ? -INFINITY : (from_base + log2f(l)) * kLn2;
}

constexpr int kBothBytes = std::max(2 * own::kPlace, prefix::kBytes);
static_assert(kBothBytes <= 227 * 1024 && kResident * (own::kBytes + 1024) <= 228 * 1024, "what an SM has");

template <bool F16, int kEights>
cudaError_t launch(const AttentionParams& p, cudaStream_t stream) {
  static thread_local int generation = -1, device = -1;  // the attribute is one of a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (generation != launch_config_generation() || device != dev) {
    e = cudaFuncSetAttribute(gdn_attention_kernel<F16, kEights>, cudaFuncAttributeMaxDynamicSharedMemorySize, own::kBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_attention_both_kernel<F16, kEights>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBothBytes);
    if (e != cudaSuccess) return e;
    generation = launch_config_generation();
    device = dev;
  }
  const int64_t subs = (int64_t)p.H_k * p.blocks, own_units = p.N * subs;
  const int64_t most = ((int64_t)p.max_pages * p.page_size + kOwnKeys - 1) / kOwnKeys * own_units +
                       ((int64_t)p.prefix + kOwnKeys - 1) / kOwnKeys * p.H_k * p.prefix_blocks;
  const bool many = p.prefix_units > 0;
  if (many) e = launch_behind(gdn_attention_both_kernel<F16, kEights>, p.prefix_workers, prefix::kThreads, kBothBytes, stream, p);
  else if (most) e = launch_behind(gdn_attention_kernel<F16, kEights>, std::min<int64_t>(p.workers, most), own::kThreads, own::kBytes, stream, p);
  if (e != cudaSuccess) return e;
  // Warps a row by the parts that a row has about, as long as the rows' CTAs find a place all at once (three of eight warps or one of 32
  // an SM); after that rows keep the SMs busy with a warp each.  us of a call with 32 warps, 8 warps, a warp by sixes and by eights:
  //   153 parts, 16 rows      27 28 46 47      184 parts, 160 rows     27 29 90 64      31 parts, 160 rows      19 17 24 23
  //   77 parts, 64 rows       26 27 37 36      49 parts, 256 rows      48 47 58 52      10 parts, 512 rows      109.5 105.4 106.3 105.6
  //   192 parts, 128 rows     20 26 87 57      45 parts, 448 rows      53 48 59 54      5 parts, 512 rows       51 47 45 46
  //   39 parts, 32 rows       86 87 91 90      43 parts, 640 rows      61 53 62 56      3 parts, 1332 rows      37 26 24 23
  const int64_t prefix_tiles = ((int64_t)p.prefix + kPrefixKeys - 1) / kPrefixKeys, sms = p.workers / kResident;
  int64_t parts = 1 + p.workers / (own_units + p.H_k * p.prefix_blocks);
  if (many) parts += 1 + std::min<int64_t>(prefix_tiles - 1, p.prefix_workers / ((int64_t)p.H_k * p.prefix_units));
  const int64_t rows = own_units * p.block_rows;
  if (parts > 64 && rows <= sms) return launch_behind(gdn_attention_join_kernel<F16, 32, 5>, rows, kJoinThreads<32>, 0, stream, p);
  if (parts > 8 && rows <= 3 * sms) return launch_behind(gdn_attention_join_kernel<F16, 8, 8>, rows, kJoinThreads<8>, 0, stream, p);
  // Few parts a row leave room for more rows instead: 8192 rows of 6 parts take 1.3 us less by sixes than by eights, 3888 of 12 1.5 us less;
  // 512 of 44 5 us more, 564 of 58 2 us more.
  if (parts <= 12) return launch_behind(gdn_attention_join_kernel<F16, 1, 6>, (rows + 3) / 4, kJoinThreads<1>, 0, stream, p);
  return launch_behind(gdn_attention_join_kernel<F16, 1, 8>, (rows + 3) / 4, kJoinThreads<1>, 0, stream, p);
}

}  // namespace

size_t plan_attention(AttentionParams* p, int sms, void* workspace) {
  p->group = p->H_q / p->H_k;
  const int64_t rows = (int64_t)p->tokens * p->group, all = p->N * rows;
  // More than a block's rows a key head go to the tensor cores, whatever the prefix' length.  8 rows of 2 key heads and 30000 keys take
  // 14.4 us there and 12.8 us in the walk, 16 rows of 8 heads 32.6 and 34.8 us, 256 rows of 4 heads and 64 keys 14.4 and 14.3 us,
  // 8192 keys 23 and 40 us (with 300 keys of its own a sequence).
  const bool many = p->prefix && all > own::kRows;
  p->workers = kResident * sms;
  p->blocks = (int32_t)((rows + own::kRows - 1) / own::kRows);
  p->block_groups = (p->blocks + 3) / 4;   // L2 feeds some two to three times what HBM does, so more side by side gain nothing
  p->blocks_aside = (p->blocks + p->block_groups - 1) / p->block_groups;
  p->prefix_blocks = p->prefix && !many ? 1 : 0;
  p->block_rows = (int32_t)std::min<int64_t>(own::kRows, p->prefix_blocks ? all : rows);
  p->prefix_units = many ? (int32_t)((all + kPrefixRows - 1) / kPrefixRows) : 0;
  const int64_t many_units = (int64_t)p->H_k * p->prefix_units;
  p->prefix_workers = many ? sms : 0;   // or fewer: the device shares the SMs out
  p->by_group = divisor(p->group);
  p->by_page = divisor(p->page_size);
  p->by_groups = divisor(p->block_groups);
  p->by_rows = divisor(p->block_rows);
  p->by_blocks = divisor(p->blocks);
  p->by_aside = divisor(p->blocks_aside);
  p->by_subs = divisor(p->H_k * p->blocks);
  p->by_units = divisor(p->prefix_units);
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
  int32_t* first_worker = reinterpret_cast<int32_t*>(take((size_t)(units + many_units) * 8));
  if (workspace) {
    p->part_o = part_o; p->part_ml = part_ml;
    p->prefix_o = prefix_o; p->prefix_ml = prefix_ml;
    p->first_worker = first_worker; p->last_worker = first_worker + units;
    p->prefix_first = first_worker + 2 * units; p->prefix_last = p->prefix_first + many_units;
  }
  return end;
}

cudaError_t launch_attention(const AttentionParams& p, cudaStream_t stream) {
  if (p.block_rows <= 8) return p.op_f16 ? launch<true, 1>(p, stream) : launch<false, 1>(p, stream);
  return p.op_f16 ? launch<true, 2>(p, stream) : launch<false, 2>(p, stream);
}

}  // namespace gdn
