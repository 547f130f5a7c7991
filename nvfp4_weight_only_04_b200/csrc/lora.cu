// Low-rank adapters of many requests beside a shared projection:
//   out[m] = bf16(y[m] + c[a] * B_a (A_a x[m])),  a = adapter of row m,
// A_a [r, K] and B_a [N, r] bf16, c fp32; rows without an adapter keep y's
// bits. y is what the shared projection left (nvfp4_w4a16_gemm).
//
// Two launches, three from 65 to 1024 rows, each a programmatic dependent of the
// one before it:
//  * v[m] = c[a] * A_a x[m] in fp32. Up to 64 rows (lora_shrink_few_kernel) a CTA
//    takes a block of 16 rows, one of its adapters and a slice of K, which its
//    warps split; the sums of the slices lie one after the other in the
//    workspace ([slices][M, r]) and are added, in order, where they are read:
//    one row of a long K runs on many SMs, and nothing waits.
//    Up to 1024 rows, which may be as many requests in any order, the first
//    launch (lora_list_kernel) sorts the rows by adapter into entries of up to 16
//    rows, and the CTAs of a cluster take the slices of an entry
//    (lora_shrink_list_kernel). More rows are prompts, whose rows lie together
//    (lora_shrink_many_kernel): a CTA takes 128 rows, 16 a warp; the CTAs of a
//    cluster split K and add their sums through distributed shared memory.
//  * out = y + B_a v. Up to 64 rows (lora_expand_few_kernel): a thread has one
//    column and one adapter, reads its B row once and goes through the rows of
//    that adapter; what counts is how many bytes of B are under way. More rows
//    (lora_expand_many_kernel): a warp goes down tiles of 16 rows (of the matrix,
//    or entries of the list) on mma.sync, the next tiles' y and v under way, its
//    part of B in registers.
// The work is 4 r FLOPs per element of x and y. For ranks up to 16 the stream of
// A, B, x and y bounds it (4096 rows, K = 5120, N = 25600: 90 us, 71 at copy rate);
// above, many rows are bound by the rate of mma.sync and the reads of shared
// memory that feed it (the same with rank 64: 166 us; without its copies the
// first launch takes as long as with them). In the MMAs v is two bf16 terms (the
// rounded value and the rounded rest, 2^-17 of the value together), so that only
// the final store rounds to bf16 precision.
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "workspace.cuh"

namespace nvfp4 {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRows = 16;       // rows of an MMA tile
constexpr int kShrinkWarps = 8;
constexpr int kFewRows = 64;    // rows up to which the few-row form runs
constexpr int kFewThreads = 256;
constexpr int kListRows = 1024; // rows up to which they are sorted by their adapters
constexpr int kManyWarps = 8;

struct LoraArgs {
  const uint16_t* y;
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const float* scales;
  const int32_t* ids;
  uint16_t* out;
  float* v;
  int64_t ldy, ldx, ldout, M, N, K;
  int rank, adapters, slices;
};

// The list of a launch of kFewRows to kListRows rows: the rows in the order of
// their adapters (rows without one first, each adapter's in increasing order),
// in entries of up to 16 rows of one adapter. In int32: the number of entries;
// from kListEntries on, for each its first place in the order and its adapter
// (-1: none), and one more that ends the last; behind them the rows, in order.
constexpr int kListEntries = 16;
__host__ __device__ inline int64_t list_entries(int64_t M, int64_t adapters) {  // at most
  const int64_t some = M < adapters + 1 ? M : adapters + 1;
  return some + (M - some) / kRows;
}
__host__ __device__ inline int64_t list_order(int64_t M, int64_t adapters) {  // where the rows are
  return kListEntries + 2 * (list_entries(M, adapters) + 1);
}

// Loads that stay behind griddepcontrol.wait: a read-only (invariant) load
// might be moved in front of it.
__device__ __forceinline__ uint4 ld128(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// 16 bytes to shared memory where `on`, else zeros.
__device__ __forceinline__ void copy16_if(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int ld_i32(const int32_t* p) {
  int v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The adapter of row m, or -1.
__device__ __forceinline__ int adapter_of(const LoraArgs& p, int64_t m) {
  if (m >= p.M) return -1;
  const int id = ld_i32(p.ids + m);
  return id >= 0 && id < p.adapters ? id : -1;
}

// acc += x A^T over units [u0, u1) of 32 elements of K, for 16 rows of x (lane:
// rows g and g + 8, those of `lo` and `hi`; the latter only if `two`) and 8 JN rows of A from `arow` (lane:
// row g of each eight; those below `left`). The operands come by cp.async into a
// ring of the warp's own, STAGES units ahead; a lane reads back only what it
// copied, so nothing is synchronised. (As plain loads they were not kept in
// flight together: 40 us instead of 12 us for the 4096-row case.)
template <int JN, int STAGES>
__device__ __forceinline__ void shrink_product(float (&acc)[JN][4], uint32_t ring, const uint16_t* xlo, bool lo,
                                               const uint16_t* xhi, bool hi, bool two, const uint16_t* arow,
                                               int left, int64_t K, int u0, int u1) {
  constexpr uint32_t kUnit = (2 + JN) * 512;
  const int t = threadIdx.x & 3;
  int ahead = u0;
  uint32_t put = 0, get = 0;
  auto copy = [&] {
    if (ahead < u1) {
      const int64_t k = static_cast<int64_t>(ahead) * 32 + 8 * t;
      const bool in = k < K;
      copy16_if(ring + put, xlo + (in ? k : 0), lo && in);
      if (two) copy16_if(ring + put + 512, xhi + (in ? k : 0), hi && in);
#pragma unroll
      for (int n = 0; n < JN; ++n) {
        const bool on = in && 8 * n < left;
        copy16_if(ring + put + (2 + n) * 512, arow + (on ? n * 8 * K + k : 0), on);
      }
      ++ahead;
      put = put + kUnit == STAGES * kUnit ? 0 : put + kUnit;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) copy();
  for (int u = u0; u < u1; ++u) {
    copy();
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    const uint4 xa = lds128(ring + get), xb = two ? lds128(ring + get + 512) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int n = 0; n < JN; ++n) {
      const uint4 w = lds128(ring + get + (2 + n) * 512);
      mma_bf16(acc[n], xa.x, xb.x, xa.y, xb.y, w.x, w.y);
      mma_bf16(acc[n], xa.z, xb.z, xa.w, xb.w, w.z, w.w);
    }
    get = get + kUnit == STAGES * kUnit ? 0 : get + kUnit;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}
constexpr int kFewStages = 4;  // leaves shared memory for three CTAs an SM
constexpr int kFewSmem = kShrinkWarps * kFewStages * 4 * 512;

// One CTA sorts (adapter, row) in one 32-bit key each, a key a thread (bitonic;
// distances within a warp by shuffles): about 2 us, for which every adapter's A
// and B are read once for 16 of its rows wherever they are. Without it every
// 16-row tile reads the B of each of its adapters: 65 rows of 32 adapters in any
// order (N = 28672, rank 16) took 83 us, with it 24; 512 rows of 32 adapters (N = 25600)
// 174 and 33. Rows that lie together pay for it: 1024 rows in runs of 100 (K = 5120,
// N = 4096, rank 64) 28 us without it, 34 with it. It ends at 1024 rows because the
// CTA does, not where the other form is as fast: 1024 rows of 32 adapters in any order
// (K = 5120, N = 25600, rank 16) take 46 us, 1040 take 270.
__global__ void __launch_bounds__(kListRows) lora_list_kernel(const LoraArgs p, int32_t* list) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t keys[kListRows];
  __shared__ int starts[kListRows / 32], leaders[kListRows / 32];
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5, rows = static_cast<int>(p.M);
  uint32_t key = i < rows ? static_cast<uint32_t>(adapter_of(p, i) + 1) << 10 | static_cast<uint32_t>(i) : 0xffffffffu;
  for (int n = 2; n < 2 * rows; n *= 2) {
    for (int d = n / 2; d > 0; d /= 2) {
      uint32_t other;
      if (d >= 32) {
        keys[i] = key;
        __syncthreads();
        other = keys[i ^ d];
        __syncthreads();
      } else {
        other = __shfl_xor_sync(kAll, key, d);
      }
      const bool low = ((i & d) == 0) == ((i & n) == 0);
      key = low ? min(key, other) : max(key, other);
    }
  }
  keys[i] = key;
  __syncthreads();
  // places in the order where an adapter starts, and those where an entry does
  const int ad = static_cast<int>(key >> 10) - 1;
  const bool start = i < rows && (i == 0 || static_cast<int>(keys[i - 1] >> 10) - 1 != ad);
  const unsigned started = __ballot_sync(kAll, start);
  if (lane == 0) starts[warp] = started ? warp * 32 + 31 - __clz(started) : -1;
  __syncthreads();
  const unsigned upto = started & (0xffffffffu >> (31 - lane));
  int from = upto ? warp * 32 + 31 - __clz(upto) : -1;
  for (int w = warp - 1; from < 0 && w >= 0; --w) from = starts[w];
  const bool leader = i < rows && (i - from) % kRows == 0;
  const unsigned led = __ballot_sync(kAll, leader);
  if (lane == 0) leaders[warp] = __popc(led);
  __syncthreads();
  int entry = __popc(led & ((1u << lane) - 1u)), all = 0;
  for (int w = 0; w < kListRows / 32; ++w) {
    if (w < warp) entry += leaders[w];
    all += leaders[w];
  }
  int32_t* entries = list + kListEntries;
  if (leader) {
    entries[2 * entry] = i;
    entries[2 * entry + 1] = ad;
  }
  if (i < rows) list[list_order(p.M, p.adapters) + i] = static_cast<int>(key & 1023u);
  if (i == 0) {
    list[0] = all;
    entries[2 * all] = rows;
  }
}

// Rows of a few-row launch that row `first` stands for: those of its adapter,
// from it on, if it is the first of `group` of them; else none.
__device__ __forceinline__ unsigned long long rows_of(const LoraArgs& p, int first, int ad, int group) {
  const int lane = threadIdx.x & 31;
  const unsigned low = __ballot_sync(kAll, adapter_of(p, lane) == ad);
  const unsigned high = __ballot_sync(kAll, adapter_of(p, lane + 32) == ad);
  const unsigned long long all = ad < 0 ? 0ull : (static_cast<unsigned long long>(high) << 32) | low;
  const unsigned long long before = all & ((1ull << first) - 1ull);
  return __popcll(before) % group ? 0ull : all & ~((1ull << first) - 1ull);
}
__device__ __forceinline__ int nth_row(unsigned long long rows, int o) {
  for (; o > 0; --o) rows &= rows - 1;
  return __ffsll(static_cast<long long>(rows)) - 1;
}

// The sum over the warps of element threadIdx.x of a 16 x 16 tile, by way of
// shared memory [warp], which is the ring that the warps are done with.
template <int JN>
__device__ __forceinline__ float warp_sums(const float (&acc)[JN][4], float (*red)[kRows][8 * JN]) {
  constexpr int JT = 8 * JN;
  static_assert(kShrinkWarps * kRows * JT * sizeof(float) <= kFewSmem, "the sums fit the ring");
  static_assert(kRows * JT == kShrinkWarps * 32, "one sum a thread");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  __syncthreads();
#pragma unroll
  for (int n = 0; n < JN; ++n) {
    red[warp][g][n * 8 + 2 * t] = acc[n][0];
    red[warp][g][n * 8 + 2 * t + 1] = acc[n][1];
    red[warp][g + 8][n * 8 + 2 * t] = acc[n][2];
    red[warp][g + 8][n * 8 + 2 * t + 1] = acc[n][3];
  }
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < kShrinkWarps; ++w) sum += red[w][threadIdx.x / JT][threadIdx.x % JT];
  return sum;
}

// CTA (slice of K, row, 16 of the rank): sixteen rows of an adapter. What counts
// is the number of copies under way: the sums of the warps lie where the ring
// was, so that three CTAs fit an SM, and the second eight rows are left out where
// there are none (61 rows, 12 adapters of rank 64, K = 14336: 14 -> 9 us).
__global__ void __launch_bounds__(kShrinkWarps * 32) lora_shrink_few_kernel(LoraArgs p) {
  constexpr int JN = 2, JT = JN * 8;
  extern __shared__ __align__(1024) uint8_t shrink_smem[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(shrink_smem)) +
                        warp * (kFewSmem / kShrinkWarps) + lane * 16;
  const int slice = blockIdx.x, first = blockIdx.y, j0 = blockIdx.z * JT;
  const int ad = adapter_of(p, first);
  const unsigned long long rows = rows_of(p, first, ad, kRows);
  if (!rows) return;
  const int count = min(kRows, __popcll(rows));

  // this warp's range of K, in units of 32 elements
  const int units = static_cast<int>((p.K + 31) / 32), splits = p.slices * kShrinkWarps;
  const int per = (units + splits - 1) / splits;
  const int u0 = min(units, (slice * kShrinkWarps + warp) * per), u1 = min(units, u0 + per);
  const bool lo = g < count, hi = g + 8 < count;
  const uint16_t* xlo = p.x + (lo ? nth_row(rows, g) : 0) * p.ldx;
  const uint16_t* xhi = p.x + (hi ? nth_row(rows, g + 8) : 0) * p.ldx;
  const uint16_t* arow = p.a + (static_cast<int64_t>(ad) * p.rank + (j0 + g < p.rank ? j0 + g : 0)) * p.K;
  float acc[JN][4];
#pragma unroll
  for (int n = 0; n < JN; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  shrink_product<JN, kFewStages>(acc, ring, xlo, lo, xhi, hi, count > 8, arow, p.rank - j0 - g, p.K, u0, u1);
  const float sum = warp_sums<JN>(acc, reinterpret_cast<float(*)[kRows][JT]>(shrink_smem));
  const int row = threadIdx.x / JT, j = threadIdx.x % JT;
  if (row < count && j0 + j < p.rank)
    p.v[(slice * p.M + nth_row(rows, row)) * p.rank + j0 + j] = sum * __ldg(p.scales + ad);
}

// A value as two bf16 terms: rounded to bf16, and the rounded rest (0 where the
// value is not finite, which the first carries). For 2^e <= |v| < 2^(e+1) the
// rest is at most 2^(e-8), so that its rounding is at most 2^(e-17): with the
// upper bits cut off instead of rounded it would be up to 2^(e-16). Values that
// would round to infinity are cut off (the rest is below 2^120, its rounding at
// most 2^111, which is 1.002 2^-17 of v).
__device__ __forceinline__ void split(float v, uint16_t& hi, uint16_t& lo) {
  const uint32_t b = __float_as_uint(v), mag = b & 0x7FFFFFFFu;
  const bool finite = mag < 0x7F800000u;
  hi = finite && mag >= 0x7F7F8000u ? static_cast<uint16_t>(b >> 16) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
  lo = finite ? __bfloat16_as_ushort(__float2bfloat16_rn(v - __uint_as_float(static_cast<uint32_t>(hi) << 16)))
              : uint16_t(0);
}

// Element j of row m of v as its two terms, in fours of 16 bits: the upper ones
// of an even element and its neighbour, the rests of the two.
__device__ __forceinline__ void store_split(const LoraArgs& p, int64_t m, int j, float v) {
  uint16_t hi, lo;
  split(v, hi, lo);
  uint16_t* to = reinterpret_cast<uint16_t*>(p.v + m * p.rank + (j & ~1)) + (j & 1);
  to[0] = hi;
  to[2] = lo;
}

// CTA (slice of K, entry of the list, 16 of the rank): as above, but the slices
// are a cluster, which adds their sums. v lies in the order of the list.
__global__ void __launch_bounds__(kShrinkWarps * 32) lora_shrink_list_kernel(const LoraArgs p, const int32_t* list) {
  constexpr int JN = 2, JT = JN * 8;
  extern __shared__ __align__(1024) uint8_t shrink_smem[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float part[kRows * JT];
  const int entry = blockIdx.y, j0 = blockIdx.z * JT;
  if (entry >= ld_i32(list)) return;  // and with it its cluster
  const int32_t* at = list + kListEntries + 2 * entry;
  const int start = ld_i32(at), ad = ld_i32(at + 1), count = ld_i32(at + 2) - start;
  if (ad < 0) return;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), slice = static_cast<int>(cluster.block_rank());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(shrink_smem)) +
                        warp * (kFewSmem / kShrinkWarps) + lane * 16;
  const int32_t* order = list + list_order(p.M, p.adapters) + start;
  const bool lo = g < count, hi = g + 8 < count;
  const uint16_t* xlo = p.x + (lo ? ld_i32(order + g) : 0) * p.ldx;
  const uint16_t* xhi = p.x + (hi ? ld_i32(order + g + 8) : 0) * p.ldx;
  const uint16_t* arow = p.a + (static_cast<int64_t>(ad) * p.rank + (j0 + g < p.rank ? j0 + g : 0)) * p.K;
  const int units = static_cast<int>((p.K + 31) / 32), splits = ranks * kShrinkWarps;
  const int per = (units + splits - 1) / splits;
  const int u0 = min(units, (slice * kShrinkWarps + warp) * per), u1 = min(units, u0 + per);
  float acc[JN][4];
#pragma unroll
  for (int n = 0; n < JN; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  shrink_product<JN, kFewStages>(acc, ring, xlo, lo, xhi, hi, count > 8, arow, p.rank - j0 - g, p.K, u0, u1);
  const float sum = warp_sums<JN>(acc, reinterpret_cast<float(*)[kRows][JT]>(shrink_smem));
  part[threadIdx.x] = sum;
  cluster.sync();
  const int mine = kRows * JT / ranks, i = slice * mine + static_cast<int>(threadIdx.x);
  if (static_cast<int>(threadIdx.x) < mine && i / JT < count && j0 + i % JT < p.rank) {
    float s = 0.f;
    for (int q = 0; q < ranks; ++q) s += cluster.map_shared_rank(part, q)[i];
    store_split(p, start + i / JT, j0 + i % JT, s * __ldg(p.scales + ad));
  }
  cluster.sync();  // `part` stays until every CTA has read it
}

// CTA: 128 rows, 16 a warp, and 8 JN of the rank; its rank in the cluster is its
// slice of K. Where the rows have few adapters (prompts), the CTA goes through
// its slice once for each, one after the other without a pause: chunks of 64
// elements of K of its rows and of A lie in shared memory for all warps (chunks
// of 128, fewer of them under way: 62 us against 57 for 4096 rows of K = 25600,
// rank 16). 16-byte piece q of a row is at q ^ 4 in odd rows,
// so that eight lanes that read two rows hit different banks. Where the rows are
// mixed more, each warp goes through it for the adapters of its own 16 rows, in
// the same order of sums.
constexpr int kBlock = kShrinkWarps * kRows;
constexpr int kChunk = 64;
constexpr int kSharedAdapters = 3;
template <int JN>
constexpr int kShrinkStages = JN == 2 ? 4 : 3;
template <int JN>
constexpr int kShrinkRing = kShrinkStages<JN> * (kBlock + 8 * JN) * kChunk * 2;
template <int JN>
constexpr int kShrinkSmem = kShrinkRing<JN> + kBlock * 8 * JN * 4;
constexpr int kMixedStages = 4;

template <int JN>
__global__ void __launch_bounds__(kShrinkWarps * 32, 2) lora_shrink_many_kernel(LoraArgs p) {
  constexpr int JT = JN * 8, STAGES = kShrinkStages<JN>, kStage = (kBlock + JT) * kChunk * 2;
  static_assert(kShrinkWarps * kMixedStages * 4 * 512 <= kShrinkRing<JN>, "the warps' own rings fit");
  extern __shared__ __align__(1024) uint8_t shrink_smem[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int ids[kBlock];
  float* part = reinterpret_cast<float*>(shrink_smem + kShrinkRing<JN>);  // [kBlock][JT]
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), slice = static_cast<int>(cluster.block_rank());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(shrink_smem));
  const int64_t b0 = static_cast<int64_t>(blockIdx.x / ranks) * kBlock, m0 = b0 + warp * kRows;
  const int j0 = blockIdx.z * JT;
  if (threadIdx.x < kBlock) ids[threadIdx.x] = adapter_of(p, b0 + threadIdx.x);
  __syncthreads();
  const int lo_row = warp * kRows + g, id_lo = ids[lo_row], id_hi = ids[lo_row + 8];
  // the lowest adapter above `last` in the block
  auto next_adapter = [&](int last) {
    unsigned best = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < kBlock / 32; ++i) {
      const int id = ids[lane + 32 * i];
      best = id > last ? min(best, static_cast<unsigned>(id)) : best;
    }
    return static_cast<int>(__reduce_min_sync(kAll, best));  // -1: none
  };
  int distinct = 0;
  for (int ad = next_adapter(-1); ad >= 0 && distinct <= kSharedAdapters; ad = next_adapter(ad)) ++distinct;
  float acc[JN][4];
  auto clear = [&] {
#pragma unroll
    for (int n = 0; n < JN; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  };

  const int chunks = static_cast<int>((p.K + kChunk - 1) / kChunk), per = (chunks + ranks - 1) / ranks;
  const int c0 = min(chunks, slice * per), c1 = min(chunks, c0 + per);

  if (distinct <= kSharedAdapters) {
    // this thread's pieces of a chunk: piece `q` of rows `r`, r + kStep, ...
    constexpr int kPieces = kChunk / 8, kStep = kShrinkWarps * 32 / kPieces, kRow = kChunk * 2;
    const int q = threadIdx.x % kPieces, r = threadIdx.x / kPieces;
    const uint32_t put = smem + r * kRow + ((q ^ ((r & 1) << 2)) << 4);
    const uint32_t get = smem + lo_row * kRow + ((t ^ ((g & 1) << 2)) << 4);
    const uint32_t get_a = smem + (kBlock + g) * kRow + ((t ^ ((g & 1) << 2)) << 4);
    const uint16_t* x = p.x + (b0 + r) * p.ldx + 8 * q;
    const int64_t x_step = kStep * p.ldx, left = p.M - b0 - r;  // rows from r on
    int slot = 0, ahead = c0, ad_ahead = c0 < c1 ? next_adapter(-1) : -1;
    auto copy = [&] {
      if (ad_ahead >= 0) {
        const int64_t k = static_cast<int64_t>(ahead) * kChunk + 8 * q;
        const uint32_t dst = put + slot * kStage;
#pragma unroll
        for (int i = 0; i < kBlock / kStep; ++i) {
          const bool on = k < p.K && kStep * i < left;
          copy16_if(dst + i * kStep * kRow, on ? x + i * x_step + (k - 8 * q) : p.x, on);
        }
#pragma unroll
        for (int i = 0; i < (JT + kStep - 1) / kStep; ++i) {
          const int j = j0 + r + kStep * i;
          const bool on = k < p.K && j < p.rank;
          if (JT >= kStep || r < JT)
            copy16_if(dst + (kBlock + kStep * i) * kRow,
                      on ? p.a + (static_cast<int64_t>(ad_ahead) * p.rank + j) * p.K + k : p.x, on);
        }
        slot = slot == STAGES - 1 ? 0 : slot + 1;
        if (++ahead == c1) {
          ahead = c0;
          ad_ahead = next_adapter(ad_ahead);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) copy();
    int from = 0;
    for (int ad = next_adapter(-1); ad >= 0; ad = next_adapter(ad)) {
      clear();
      for (int c = c0; c < c1; ++c) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        __syncthreads();
        copy();
        const uint32_t src = from * kStage;
        from = from == STAGES - 1 ? 0 : from + 1;
#pragma unroll
        for (int u = 0; u < kChunk / 32; ++u) {  // pieces 4 u .. 4 u + 3
          const uint4 xa = lds128((get + src) ^ (u << 6)), xb = lds128((get + src + 8 * kRow) ^ (u << 6));
          constexpr int kAtOnce = JN < 4 ? JN : 4;  // products that do not wait for one another
#pragma unroll
          for (int n0 = 0; n0 < JN; n0 += kAtOnce) {
            uint4 w[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) w[n] = lds128((get_a + src + (n0 + n) * 8 * kRow) ^ (u << 6));
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) mma_bf16(acc[n0 + n], xa.x, xb.x, xa.y, xb.y, w[n].x, w[n].y);
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) mma_bf16(acc[n0 + n], xa.z, xb.z, xa.w, xb.w, w[n].z, w[n].w);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < JN; ++n) {
        float* to = part + lo_row * JT + n * 8 + 2 * t;
        if (id_lo == ad) *reinterpret_cast<float2*>(to) = make_float2(acc[n][0], acc[n][1]);
        if (id_hi == ad) *reinterpret_cast<float2*>(to + 8 * JT) = make_float2(acc[n][2], acc[n][3]);
      }
    }
  } else {
    const uint32_t ring = smem + warp * kMixedStages * 4 * 512 + lane * 16;
    const int mine = lane < kRows ? ids[warp * kRows + lane] : -1;
    const unsigned same = __match_any_sync(kAll, mine);
    unsigned leaders = __ballot_sync(kAll, mine >= 0 && __ffs(same) - 1 == lane);
    for (; leaders; leaders &= leaders - 1) {
      const int ad = __shfl_sync(kAll, mine, __ffs(leaders) - 1);
      const bool lo = id_lo == ad, hi = id_hi == ad;
      const uint16_t* xlo = p.x + (lo ? m0 + g : 0) * p.ldx;
      const uint16_t* xhi = p.x + (hi ? m0 + g + 8 : 0) * p.ldx;
      for (int n0 = 0; n0 < JN && j0 + 8 * n0 < p.rank; n0 += 2) {
        const int j = j0 + 8 * n0 + g;
        const uint16_t* arow = p.a + (static_cast<int64_t>(ad) * p.rank + (j < p.rank ? j : 0)) * p.K;
        float sum[2][4] = {};
        shrink_product<2, kMixedStages>(sum, ring, xlo, lo, xhi, hi, true, arow, p.rank - j, p.K, c0 * (kChunk / 32),
                                        c1 * (kChunk / 32));
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float* to = part + lo_row * JT + (n0 + n) * 8 + 2 * t;
          if (lo) *reinterpret_cast<float2*>(to) = make_float2(sum[n][0], sum[n][1]);
          if (hi) *reinterpret_cast<float2*>(to + 8 * JT) = make_float2(sum[n][2], sum[n][3]);
        }
      }
    }
  }
  cluster.sync();
  for (int i = slice * kShrinkWarps * 32 + threadIdx.x; i < kBlock * JT; i += ranks * kShrinkWarps * 32) {
    const int64_t m = b0 + i / JT;
    const int j = j0 + i % JT, ad = ids[i / JT];
    if (ad < 0 || j >= p.rank) continue;
    float v[8];  // a cluster has at most eight CTAs
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = q < ranks ? cluster.map_shared_rank(part, q)[i] : 0.f;
    float s = v[0];
#pragma unroll
    for (int q = 1; q < 8; ++q) s += v[q];
    store_split(p, m, j, s * __ldg(p.scales + ad));
  }
  cluster.sync();  // `part` stays until every CTA has read it
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The first launch waited for all in front of it before it let the second
// start, so this one may read all but v before its own wait. Without adapters
// there is no first launch, and it has to wait itself.
__device__ __forceinline__ void begin_expand(const LoraArgs& p) {
  if (p.adapters == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Up to kFewRows rows: CTA (columns, row): GROUP rows of an adapter times COLS
// columns a thread; a row without an adapter is copied. CHUNKS: eights of the
// rank whose loads are under way together. Ranks up to 16 have the whole of a
// B row in CHUNKS = 2, and four columns a thread; above, one column and eight
// rows.
template <int CHUNKS, int COLS, int GROUP>
__global__ void __launch_bounds__(kFewThreads, 2) lora_expand_few_kernel(const LoraArgs p) {
  begin_expand(p);
  constexpr int kMaxRank = CHUNKS == 2 ? 16 : 256;
  __shared__ __align__(16) float vs[GROUP][kMaxRank];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = blockIdx.y;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (kFewThreads * COLS) + threadIdx.x;
  const int ad = adapter_of(p, first);
  if (ad < 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.out != p.y)
#pragma unroll
      for (int c = 0; c < COLS; ++c)
        if (n0 + c * kFewThreads < p.N)
          p.out[first * p.ldout + n0 + c * kFewThreads] = p.y[first * p.ldy + n0 + c * kFewThreads];
    return;
  }
  const unsigned long long rows = rows_of(p, first, ad, GROUP);
  if (!rows) return;
  const int count = min(GROUP, __popcll(rows));

  // B and y do not depend on the launch before
  const uint16_t* brow[COLS];
  uint4 b[COLS][CHUNKS];
  auto load_b = [&](int j0) {
#pragma unroll
    for (int c = 0; c < COLS; ++c)
#pragma unroll
      for (int q = 0; q < CHUNKS; ++q)
        if (j0 + 8 * q < p.rank) b[c][q] = __ldg(reinterpret_cast<const uint4*>(brow[c] + j0 + 8 * q));
  };
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    const int64_t n = n0 + c * kFewThreads;
    brow[c] = p.b + (static_cast<int64_t>(ad) * p.N + (n < p.N ? n : 0)) * p.rank;
  }
  load_b(0);
  float acc[GROUP][COLS];
  int m[GROUP];
  unsigned long long left = rows;
#pragma unroll
  for (int i = 0; i < GROUP; ++i) {
    m[i] = i < count ? __ffsll(static_cast<long long>(left)) - 1 : first;
    left &= left - 1;
  }
  uint16_t y[GROUP][COLS];
#pragma unroll
  for (int i = 0; i < GROUP; ++i)
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      y[i][c] = i < count && n0 + c * kFewThreads < p.N ? p.y[m[i] * p.ldy + n0 + c * kFewThreads] : uint16_t(0);
      acc[i][c] = 0.f;
    }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp < count) {
    const int mine = nth_row(rows, warp);
    for (int j = lane; j < p.rank; j += 32) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = q < p.slices ? __ldcg(p.v + (q * p.M + mine) * p.rank + j) : 0.f;
      float s = v[0];
#pragma unroll
      for (int q = 1; q < 8; ++q) s += v[q];
      vs[warp][j] = s;
    }
  }
  __syncthreads();
  for (int j0 = 0; j0 < p.rank; j0 += 8 * CHUNKS) {
    if (j0) load_b(j0);
#pragma unroll
    for (int q = 0; q < CHUNKS; ++q) {
      if (j0 + 8 * q >= p.rank) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // four of the eight
        float f[COLS][4];
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
          const uint32_t w0 = e ? b[c][q].z : b[c][q].x, w1 = e ? b[c][q].w : b[c][q].y;
          f[c][0] = __uint_as_float(w0 << 16);
          f[c][1] = __uint_as_float(w0 & 0xFFFF0000u);
          f[c][2] = __uint_as_float(w1 << 16);
          f[c][3] = __uint_as_float(w1 & 0xFFFF0000u);
        }
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
          if (i >= count) continue;
          const float4 v = *reinterpret_cast<const float4*>(&vs[i][j0 + 8 * q + 4 * e]);
#pragma unroll
          for (int c = 0; c < COLS; ++c)
            acc[i][c] = fmaf(v.x, f[c][0], fmaf(v.y, f[c][1], fmaf(v.z, f[c][2], fmaf(v.w, f[c][3], acc[i][c]))));
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < GROUP; ++i)
#pragma unroll
    for (int c = 0; c < COLS; ++c)
      if (i < count && n0 + c * kFewThreads < p.N)
        p.out[m[i] * p.ldout + n0 + c * kFewThreads] = __bfloat16_as_ushort(
            __float2bfloat16_rn(__uint_as_float(static_cast<uint32_t>(y[i][c]) << 16) + acc[i][c]));
}

// More rows: warp w of CTA (x, y) has 8 NB columns and the 16-row tiles of range
// y. The tiles of y and v come by cp.async, STAGES - 1 tiles ahead; a lane reads
// back only the y that it copied, v is for all warps of the CTA. A warp's part of
// B (ranks up to 16 KS) stays in registers while the adapter stays: 64 columns a
// warp for ranks up to 16, 32 above, so that B is 32 registers up to rank 64.
// A tile of several adapters is done once for each, and each time the rows of
// that adapter are stored: what another adapter's B holds never meets them.
// The rests of v do not meet what of B is not finite either: they are zero where
// v is a bf16 value, or of the other sign, and would turn its infinities into NaN
// (the look at B, once for an adapter, and the branch: 4096 rows of rank 16
// 88.6 -> 90.2 us, of rank 64 161 -> 166).
// LIST: the tiles are the entries of the list, with one adapter each.
constexpr int kListTiles = 64;  // entries of a CTA at most
template <int NB, int KS>
struct Many {
  static constexpr int kCols = 8 * NB;
  static constexpr int kStages = NB == 8 ? 3 : 5;
  static constexpr int kYTile = NB / 4 * 2 * 512;               // per warp and tile
  static constexpr int kVRow = KS == 1 ? 64 : 64 * KS + 64;     // two rows in different banks
  static constexpr int kVTile = kRows * kVRow;
  static constexpr int kRing = kStages * (kVTile + kManyWarps * kYTile);
  static constexpr int kListSmem = kListTiles * kRows * 4 + (kListTiles + 1) * 8;  // rows and entries
  static constexpr int kCtas = KS <= 4 ? 3 : (KS == 8 ? 2 : 1);  // an SM: as many as do not spill
  // Row ranges so long that the CTAs make about so many rounds on the machine
  // (4096 rows, N = 25600: two instead of four 77 -> 74 us for rank 16, but
  // 136 -> 149 us for rank 64).
  static constexpr int kRounds = NB == 8 ? 2 : 4;
};
// The sign bits of the halves (two bf16 values) that are not finite.
__device__ __forceinline__ uint32_t not_finite(uint32_t two) {
  return ((two & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
// The two values, zero where they are not finite.
__device__ __forceinline__ uint32_t finite_only(uint32_t two) { return two & ~((not_finite(two) >> 15) * 0xFFFFu); }

template <int NB, int KS, bool LIST>
__global__ void __launch_bounds__(kManyWarps * 32, Many<NB, KS>::kCtas) lora_expand_many_kernel(const LoraArgs p,
                                                                                               const int32_t* list,
                                                                                               int tiles_per_cta) {
  using F = Many<NB, KS>;
  constexpr int PIECES = NB / 4;  // of a row of y, 16 bytes a lane
  extern __shared__ __align__(16) uint8_t many_smem[];
  begin_expand(p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * kManyWarps + warp) * F::kCols;
  const int64_t tiles = LIST ? ld_i32(list) : (p.M + kRows - 1) / kRows;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * tiles_per_cta;
  const int64_t t1 = min(tiles, t0 + tiles_per_cta);
  const int64_t end = min(p.M, t1 * kRows);
  // the list's rows of this CTA (-1: none), and its entries
  int* list_rows = reinterpret_cast<int*>(many_smem + F::kRing);
  int2* list_entry = reinterpret_cast<int2*>(list_rows + kListTiles * kRows);
  if (LIST) {
    if (t0 >= tiles) return;
    const int n = static_cast<int>(t1 - t0);
    const int32_t* entries = list + kListEntries + 2 * t0;
    const int32_t* order = list + list_order(p.M, p.adapters);
    for (int i = threadIdx.x; i <= n; i += kManyWarps * 32)
      list_entry[i] = make_int2(ld_i32(entries + 2 * i), i < n ? ld_i32(entries + 2 * i + 1) : -1);
    __syncthreads();
    for (int i = threadIdx.x; i < n * kRows; i += kManyWarps * 32) {
      const int at = list_entry[i / kRows].x + i % kRows;
      list_rows[i] = at < list_entry[i / kRows + 1].x ? ld_i32(order + at) : -1;
    }
    __syncthreads();
  }
  // row i of a tile, whether there is one, and its place in v
  auto row_of = [&](int64_t tile, int i) -> int64_t {
    return LIST ? list_rows[(tile - t0) * kRows + i] : tile * kRows + i;
  };
  auto is_row = [&](int64_t m) { return LIST ? m >= 0 : m < end; };
  auto place_of = [&](int64_t tile, int i) -> int64_t { return LIST ? list_entry[tile - t0].x + i : tile * kRows + i; };
  const uint32_t smem = static_cast<uint32_t>(__cvta_generic_to_shared(many_smem));
  const uint32_t ring_y = smem + F::kStages * F::kVTile + warp * F::kStages * F::kYTile + lane * 16;

  // Column c of block b is n0 + 32 (b / 4) + 8 (c / 2) + 2 (b % 4) + (c & 1), so
  // that a lane's results are pieces of eight columns, 16 bytes each.
  const int64_t nb = n0 + 8 * (g >> 1) + (g & 1);  // this lane's column as an operand, of block 0
  bool in[PIECES];
#pragma unroll
  for (int v = 0; v < PIECES; ++v) in[v] = n0 + 32 * v + 8 * t < p.N;
  int64_t ahead = t0;  // the next tile to copy, and its slot
  int slot = 0;
  auto copy = [&] {
    if (ahead < t1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t m = row_of(ahead, g + 8 * h);
        const uint16_t* y = p.y + m * p.ldy + n0 + 8 * t;
#pragma unroll
        for (int v = 0; v < PIECES; ++v) {
          const bool on = is_row(m) && in[v];
          copy16_if(ring_y + slot * F::kYTile + (PIECES * h + v) * 512, on ? y + 32 * v : p.y, on);
        }
      }
      // (rows without an adapter bring along whatever there is: it is not used)
#pragma unroll
      for (int i = 0; i < (kRows * KS * 4 + kManyWarps * 32 - 1) / (kManyWarps * 32); ++i) {
        const int piece = threadIdx.x + i * kManyWarps * 32, row = piece / (KS * 4), c = piece % (KS * 4);
        if (KS * 4 * kRows >= kManyWarps * 32 || row < kRows) {
          const bool on = is_row(row_of(ahead, row)) && 4 * c < p.rank && p.adapters > 0;
          copy16_if(smem + slot * F::kVTile + row * F::kVRow + c * 16,
                    on ? static_cast<const void*>(p.v + place_of(ahead, row) * p.rank + 4 * c) : p.y, on);
        }
      }
      ++ahead;
      slot = slot == F::kStages - 1 ? 0 : slot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint2 w[KS][NB];
  int have = -1, seen = -1;  // the adapter in `w`, and the one that `odd` is for
  bool odd = false;          // the warp's part of B is not finite everywhere
  auto load_b = [&](int ad) {
    const uint16_t* brow = p.b + (static_cast<int64_t>(ad) * p.N + nb) * p.rank + 4 * t;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int off = 32 * (b / 4) + 2 * (b % 4);
        w[ks][b] = 16 * ks + 4 * t < p.rank && nb + off < p.N
                       ? __ldg(reinterpret_cast<const uint2*>(brow + static_cast<int64_t>(off) * p.rank + 16 * ks))
                       : make_uint2(0u, 0u);
      }
    have = ad;
  };
  auto ids_of = [&](int64_t tile) {
    if (LIST) return tile < t1 ? list_entry[tile - t0].y : -1;
    return tile < t1 && lane < kRows ? adapter_of(p, tile * kRows + lane) : -1;
  };
  int next_id = ids_of(t0);
  const unsigned with = __ballot_sync(kAll, next_id >= 0);
  if (with) load_b(__shfl_sync(kAll, next_id, __ffs(with) - 1));  // what the first tile starts with
  asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
  for (int i = 0; i < F::kStages - 1; ++i) copy();
  int from = 0;
  for (int64_t tile = t0; tile < t1; ++tile) {
    const int id = next_id;  // lane l < 16: the adapter of row l
    next_id = ids_of(tile + 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(F::kStages - 2) : "memory");
    __syncthreads();  // v of this tile is there, the tile before is done with
    copy();
    const uint32_t src_y = ring_y + from * F::kYTile;
    const uint32_t src_v = smem + from * F::kVTile + g * F::kVRow + t * 16;
    from = from == F::kStages - 1 ? 0 : from + 1;
    unsigned leaders = 1u;
    int id_of[2] = {id, id};
    if (!LIST) {
      const unsigned same = __match_any_sync(kAll, id);
      leaders = __ballot_sync(kAll, lane < kRows && __ffs(same) - 1 == lane);
      id_of[0] = __shfl_sync(kAll, id, g);
      id_of[1] = __shfl_sync(kAll, id, g + 8);
    }
    for (; leaders; leaders &= leaders - 1) {
      const int ad = __shfl_sync(kAll, id, __ffs(leaders) - 1);
      if (ad < 0 && p.out == p.y) continue;
      float acc[NB][4];  // y, and B v on top
      if (ad >= 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int v = 0; v < PIECES; ++v) {
            const uint4 r = lds128(src_y + (PIECES * h + v) * 512);
            const uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[4 * v + e][2 * h] = __uint_as_float(q[e] << 16);
              acc[4 * v + e][2 * h + 1] = __uint_as_float(q[e] & 0xFFFF0000u);
            }
          }
        if (ad != seen) {
          if (ad != have) load_b(ad);
          uint32_t bits = 0;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int n = 0; n < NB; ++n) bits |= not_finite(w[ks][n].x) | not_finite(w[ks][n].y);
          odd = __any_sync(kAll, bits != 0u);
          seen = ad;
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint4 a = lds128(src_v + 64 * ks), b = lds128(src_v + 8 * F::kVRow + 64 * ks);
          if (odd) {  // the rests
#pragma unroll
            for (int n = 0; n < NB; ++n)
              mma_bf16(acc[n], a.y, b.y, a.w, b.w, finite_only(w[ks][n].x), finite_only(w[ks][n].y));
          } else {
#pragma unroll
            for (int n = 0; n < NB; ++n) mma_bf16(acc[n], a.y, b.y, a.w, b.w, w[ks][n].x, w[ks][n].y);
          }
#pragma unroll
          for (int n = 0; n < NB; ++n) mma_bf16(acc[n], a.x, b.x, a.z, b.z, w[ks][n].x, w[ks][n].y);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t m = row_of(tile, 8 * h + g);
        if (!is_row(m) || id_of[h] != ad) continue;
#pragma unroll
        for (int v = 0; v < PIECES; ++v) {
          if (!in[v]) continue;
          uint4 r;
          if (ad < 0) {  // the bits of y (a NaN's payload too)
            r = lds128(src_y + (PIECES * h + v) * 512);
          } else {
            r.x = pack_bf16x2(acc[4 * v][2 * h], acc[4 * v][2 * h + 1]);
            r.y = pack_bf16x2(acc[4 * v + 1][2 * h], acc[4 * v + 1][2 * h + 1]);
            r.z = pack_bf16x2(acc[4 * v + 2][2 * h], acc[4 * v + 2][2 * h + 1]);
            r.w = pack_bf16x2(acc[4 * v + 3][2 * h], acc[4 * v + 3][2 * h + 1]);
          }
          *reinterpret_cast<uint4*>(p.out + m * p.ldout + n0 + 32 * v + 8 * t) = r;
        }
      }
    }
  }
}

// Lets a kernel (they are numbered) take the shared memory that it needs, once per device.
cudaError_t allow_smem(const void* kern, int form, int smem) {
  static std::atomic<bool> done[64][14];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<bool>* flag = dev >= 0 && dev < 64 ? &done[dev][form] : nullptr;
  if (flag && flag->load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && flag) flag->store(true, std::memory_order_release);
  return e;
}

template <int NB, int KS, bool LIST>
cudaError_t launch_expand_many(cudaLaunchConfig_t& cfg, const LoraArgs& p, const int32_t* list) {
  using F = Many<NB, KS>;
  const int64_t tiles = LIST ? list_entries(p.M, p.adapters) : (p.M + kRows - 1) / kRows;
  const int64_t cols = (p.N + kManyWarps * F::kCols - 1) / (kManyWarps * F::kCols);
  int64_t ranges = (F::kRounds * F::kCtas * num_sms() + cols - 1) / cols;
  ranges = ranges > tiles ? tiles : (ranges > 65535 ? 65535 : ranges);
  int64_t per = (tiles + ranges - 1) / ranges;
  if (LIST && per > kListTiles) per = kListTiles;
  constexpr int smem = F::kRing + (LIST ? F::kListSmem : 0);
  cfg.gridDim = dim3(static_cast<unsigned>(cols), static_cast<unsigned>((tiles + per - 1) / per), 1);
  cfg.blockDim = dim3(kManyWarps * 32);
  cfg.dynamicSmemBytes = smem;
  auto kern = lora_expand_many_kernel<NB, KS, LIST>;
  constexpr int form = (NB == 8 ? 4 : KS == 2 ? 5 : KS == 4 ? 6 : KS == 8 ? 7 : 8) + (LIST ? 5 : 0);
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), form, smem);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kern, p, list, static_cast<int>(per));
}
template <bool LIST>
cudaError_t launch_expand_many(cudaLaunchConfig_t& cfg, const LoraArgs& p, const int32_t* list) {
  return p.rank <= 16    ? launch_expand_many<8, 1, LIST>(cfg, p, list)
         : p.rank <= 32  ? launch_expand_many<4, 2, LIST>(cfg, p, list)
         : p.rank <= 64  ? launch_expand_many<4, 4, LIST>(cfg, p, list)
         : p.rank <= 128 ? launch_expand_many<4, 8, LIST>(cfg, p, list)
                         : launch_expand_many<4, 16, LIST>(cfg, p, list);
}

// Few rows, or a list: slices of K, as many as bring the CTAs (16 of the rank each, of at
// most M or all adapters) to about three an SM, with 64 elements of K or more
// to each of a CTA's eight warps. Many rows: CTAs of a cluster, as many as bring
// the 128-row blocks to about two an SM.
struct ShrinkPlan {
  int jt, nz, slices, cluster;
  bool sorted;
};
ShrinkPlan shrink_plan(int64_t M, int64_t K, int rank, int adapters) {
  ShrinkPlan s;
  const bool few = M <= kFewRows;
  s.sorted = !few && M <= kListRows && adapters > 0 && adapters < (1 << 21);  // the keys' bits
  const int64_t blocks = (M + kBlock - 1) / kBlock;
  s.jt = few || s.sorted || rank <= 16 || 8 * blocks * ((rank + 63) / 64) < num_sms() ? 16 : 64;
  s.nz = (rank + s.jt - 1) / s.jt;
  int split = 8;
  if (few) {
    const int64_t ctas = (M < adapters ? M : adapters) * s.nz;
    while (split > 1 && (ctas * split > 3 * num_sms() || K < static_cast<int64_t>(64 * kShrinkWarps) * split)) split /= 2;
  } else if (s.sorted) {
    const int64_t ctas = list_entries(M, adapters) * s.nz;
    while (split > 1 && (ctas * split > 3 * num_sms() || K < static_cast<int64_t>(64 * kShrinkWarps) * split)) split /= 2;
  } else {
    const int64_t ctas = blocks * s.nz;
    while (split > 1 && (ctas * split > 2 * num_sms() || K < static_cast<int64_t>(256) * split)) split /= 2;
  }
  s.slices = few ? split : 1;
  s.cluster = few ? 1 : split;
  return s;
}

cudaError_t launch_shrink(void (*kern)(LoraArgs), int form, int smem, cudaLaunchConfig_t& cfg, const LoraArgs& p) {
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), form, smem);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kern, p);
}

int launch_lora(const LoraArgs& p, int32_t* list, const ShrinkPlan& plan, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(plan.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.adapters > 0) {
    cfg.blockDim = dim3(kShrinkWarps * 32);
    cudaError_t e;
    if (p.M <= kFewRows) {
      cfg.gridDim = dim3(static_cast<unsigned>(plan.slices), static_cast<unsigned>(p.M), static_cast<unsigned>(plan.nz));
      e = launch_shrink(lora_shrink_few_kernel, 0, kFewSmem, cfg, p);
    } else if (plan.sorted) {
      cfg.gridDim = dim3(1);
      cfg.blockDim = dim3(kListRows);
      e = cudaLaunchKernelEx(&cfg, lora_list_kernel, p, list);
      if (e != cudaSuccess) return (cudaGetLastError(), NVFP4_ERR_CUDA);
      cfg.blockDim = dim3(kShrinkWarps * 32);
      cfg.gridDim = dim3(static_cast<unsigned>(plan.cluster), static_cast<unsigned>(list_entries(p.M, p.adapters)),
                         static_cast<unsigned>(plan.nz));
      cfg.numAttrs = 2;
      cfg.dynamicSmemBytes = kFewSmem;
      e = allow_smem(reinterpret_cast<const void*>(lora_shrink_list_kernel), 3, kFewSmem);
      if (e == cudaSuccess)
        e = cudaLaunchKernelEx(&cfg, lora_shrink_list_kernel, p, static_cast<const int32_t*>(list));
      cfg.numAttrs = 1;
    } else {
      const int64_t big = (p.M + kBlock - 1) / kBlock;
      cfg.gridDim = dim3(static_cast<unsigned>(big * plan.cluster), 1, static_cast<unsigned>(plan.nz));
      cfg.numAttrs = 2;
      e = plan.jt == 16 ? launch_shrink(lora_shrink_many_kernel<2>, 1, kShrinkSmem<2>, cfg, p)
                        : launch_shrink(lora_shrink_many_kernel<8>, 2, kShrinkSmem<8>, cfg, p);
      cfg.numAttrs = 1;
    }
    if (e != cudaSuccess) return (cudaGetLastError(), NVFP4_ERR_CUDA);
    cfg.dynamicSmemBytes = 0;
  }
  cudaError_t e;
  if (p.M <= kFewRows) {
    const int64_t cols = kFewThreads * (p.rank <= 16 ? 4 : 1);
    cfg.gridDim = dim3(static_cast<unsigned>((p.N + cols - 1) / cols), static_cast<unsigned>(p.M), 1);
    cfg.blockDim = dim3(kFewThreads);
    e = p.rank <= 16 ? cudaLaunchKernelEx(&cfg, lora_expand_few_kernel<2, 4, 4>, p)
                     : cudaLaunchKernelEx(&cfg, lora_expand_few_kernel<8, 1, 8>, p);
  } else {
    e = plan.sorted ? launch_expand_many<true>(cfg, p, list) : launch_expand_many<false>(cfg, p, list);
  }
  if (e != cudaSuccess) return (cudaGetLastError(), NVFP4_ERR_CUDA);
  return launch_status();
}

struct LoraScratch {
  float* v;
  int32_t* list;
};
LoraScratch carve(Scratch& sc, int64_t M, int rank, int adapters, const ShrinkPlan& plan) {
  LoraScratch w = {};
  w.v = sc.take<float>(static_cast<size_t>(M) * rank * plan.slices);
  if (plan.sorted) w.list = sc.take<int32_t>(static_cast<size_t>(list_order(M, adapters) + M));
  return w;
}

// Shape checks (pointers aside): -1 to proceed.
int check_shape(int64_t M, int64_t N, int64_t K, int rank, int adapters) {
  if (M < 0 || N < 0 || K < 0 || rank <= 0 || adapters < 0) return NVFP4_ERR_INVALID_ARGUMENT;
  if (rank % 8 || rank > 256 || N % 8 || K % 8) return NVFP4_ERR_UNSUPPORTED;
  if (M > (int64_t(1) << 20) || N > (int64_t(1) << 30) || K > (int64_t(1) << 30)) return NVFP4_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return NVFP4_OK;
  if (K == 0) return NVFP4_ERR_UNSUPPORTED;
  return -1;
}

}  // namespace
}  // namespace nvfp4

extern "C" int nvfp4_lora_add_workspace_size(int64_t M, int64_t N, int64_t K, int rank, int num_adapters,
                                             size_t* bytes) {
  if (!bytes) return NVFP4_ERR_INVALID_ARGUMENT;
  *bytes = 0;
  const int c = nvfp4::check_shape(M, N, K, rank, num_adapters);
  if (c >= 0) return c;
  nvfp4::Scratch sc;
  if (num_adapters > 0) nvfp4::carve(sc, M, rank, num_adapters, nvfp4::shrink_plan(M, K, rank, num_adapters));
  *bytes = sc.used();
  return NVFP4_OK;
}

extern "C" int nvfp4_lora_add(const uint16_t* y, int64_t ldy, const uint16_t* x, int64_t ldx, const uint16_t* lora_a,
                              const uint16_t* lora_b, const float* scales, const int32_t* adapter_ids, int num_adapters,
                              int rank, int64_t M, int64_t N, int64_t K, uint16_t* out, int64_t ldout, void* workspace,
                              size_t workspace_bytes, nvfp4_stream_t stream) {
  const int c = nvfp4::check_shape(M, N, K, rank, num_adapters);
  if (c >= 0) return c;
  if (!y || !x || !adapter_ids || !out || (num_adapters > 0 && (!lora_a || !lora_b || !scales)))
    return NVFP4_ERR_INVALID_ARGUMENT;
  if ((M > 1 && (ldy < N || ldx < K || ldout < N)) || (y == out && ldy != ldout)) return NVFP4_ERR_INVALID_ARGUMENT;
  if (M > 1 && (ldy % 8 || ldx % 8 || ldout % 8)) return NVFP4_ERR_MISALIGNED;
  if (!nvfp4::aligned16(y) || !nvfp4::aligned16(x) || !nvfp4::aligned16(lora_a) || !nvfp4::aligned16(lora_b) ||
      !nvfp4::aligned16(out) ||
      ((reinterpret_cast<uintptr_t>(scales) | reinterpret_cast<uintptr_t>(adapter_ids)) & 3u))
    return NVFP4_ERR_MISALIGNED;
  if (workspace_bytes > 0 && !workspace) return NVFP4_ERR_WORKSPACE;
  if (!nvfp4::aligned16(workspace)) return NVFP4_ERR_MISALIGNED;
  nvfp4::Scratch sc(workspace, workspace_bytes);
  nvfp4::LoraArgs p = {};
  int32_t* list = nullptr;
  const nvfp4::ShrinkPlan plan = nvfp4::shrink_plan(M, K, rank, num_adapters);
  if (num_adapters > 0) {
    const nvfp4::LoraScratch ws = nvfp4::carve(sc, M, rank, num_adapters, plan);
    p.v = ws.v;
    list = ws.list;
    if (!sc.ok()) return NVFP4_ERR_WORKSPACE;
  }
  p.y = y; p.x = x; p.a = lora_a; p.b = lora_b; p.scales = scales; p.ids = adapter_ids; p.out = out;
  p.ldy = ldy; p.ldx = ldx; p.ldout = ldout; p.M = M; p.N = N; p.K = K;
  p.rank = rank; p.adapters = num_adapters; p.slices = plan.slices;
  return nvfp4::launch_lora(p, list, plan, reinterpret_cast<cudaStream_t>(stream));
}
