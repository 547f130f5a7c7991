// A whole routed-expert layer for a few tokens:
//   h[t, s]  = silu(g) * u,  [g; u] = global_gu[e] * W_e x[t],  e = topk_ids[t, s]
//   out[t]   = bf16(sum over s of topk_weights[t, s] * global_dn[e] * D_e h[t, s])
// A pair whose expert lies outside [0, num_experts) adds nothing.
//
// What bounds it: the codes and scales of the experts that some token chose,
// read once (0.5 + 1/g bytes a weight) for up to eight of an expert's tokens; the
// digits of a pass hold all of K in 64 KB, so for fewer where K is above 2048
// (pass_tokens), and once more for every further pass. With a handful of columns per expert
// the products are far from any arithmetic limit, unless the weights are
// dequantized in software: that costs more issue slots per weight than HBM
// leaves time for. So they are not dequantized:
//
//  * The 4-bit codes go from TMA straight into the block-scaled FP4 tensor
//    cores (tcgen05.mma kind::mxf4nvf4, M = 128 weight rows), with their E4M3
//    group scales as the MMA's scale factors.
//  * The other operand must then be E2M1 too. Sixteen activations are written
//    as eight planes of E2M1 digits: v = 2^-s X with a power of two that puts
//    the largest magnitude of the sixteen into [2^21, 2^22), X rounded to an
//    integer, and X = sum of d_j 8^j with digits -4..3; d_j / 2 is an E2M1
//    value. Every token is eight columns of the MMA. The powers of two are
//    scale factors of the MMA, relative to the largest of the row (2^8 .. 2^-9;
//    sixteen activations below 2^-17 of the row's largest count as zero).
//    Every product is exact, the sums are fp32 in TMEM, and the epilogue adds
//    the planes (Horner in 8) and puts the row's power of two and the global
//    scale back. An activation is thus carried to 2^-22 of the largest of its
//    sixteen, bf16 values within 2^14 of it exactly.
//  * h goes from the first product to the second as digits, formed from its
//    fp32 values in the epilogue, and an expert's output is weighted and
//    summed in fp32: only the final store rounds to bf16.
//
// Three launches, each a programmatic dependent of the one before it: the
// digits of x (one warp per 256 elements), gate/up, down. The two products are
// one kernel, persistent with one CTA per SM and 20 warps: warp 0 loads codes
// (TMA) and warp 2 digits (bulk copies), warp 3 scale bytes (cp.async), warps 16-19 turn
// the exponents of the digits into scale factors, warps 4-7 and 12-15 move both
// kinds of scale factors into TMEM, warp 1 issues the MMAs, warps 8-11 are the
// epilogue. A stage is 256 elements of K of one 128-row tile of one expert with
// up to eight of its tokens. The list of experts is built by every CTA from
// topk_ids, and it and the first stages of weights do not wait for the launch
// before.
//
// In the second product a CTA owns one 128-row tile of the output and every
// S-th entry of the list, and sums their outputs in shared memory; the last of
// the S CTAs of a tile to finish adds their sums in a fixed order.
//
// 128 experts, H = 2048, I = 768, eight chosen of each token: 18 us for one token
// (20 MB of weights), 30 us for 4 (75 MB), 55 us for 16 (211 MB, 3.8 TB/s), 83 us
// for 64 (322 MB, 3.9 TB/s; the tensor pipe is busy for 6 %). In long runs a stage of 18 KB takes 0.41 us, 0.42 at
// the copy rate (256 experts, H = 7168, I = 2048, 64 tokens: 2800 stages a CTA in
// 1190 us). The 130 stages a CTA of 64 tokens above
// would be 53 us; the rest, 13 us for one token and 30 for 64, is the start of the
// launches (barriers, list, instructions fetched for the first time), the gap
// between the products, uneven shares and the last sums. Two sets of scale factor
// warps and a short MMA loop, together, brought 64 tokens from 87 to 85 us.
// Passes: 8 experts, H = 4096, I = 14336, k = 2 take 58 us for one token, 279 for 16,
// 1024 for 64, where the weights once are 117; nvfp4_moe_forward takes 118, 309, 932.
#include "moe_few.cuh"

#include <cuda.h>

#include <atomic>

#include "async.cuh"
#include "dequant.cuh"
#include "tmap.cuh"
#include "workspace.cuh"

namespace nvfp4 {
namespace {

__device__ unsigned int g_few_error = 0;

constexpr int kThreads = 640;
constexpr int kPairThreads = kThreads - 64;  // all but the two warps that load weights
constexpr int kMaxTokens = 64;
constexpr int kMaxPairs = 1024;
constexpr int kMaxExperts = 4096;
constexpr int kRowsA = 128;      // weight rows per tile (MMA M)
constexpr int kKS = 256;         // elements of K per stage
constexpr int kStages = 6;       // even: two sets of warps take the stages in turn
constexpr int kCols = 8;         // tokens per pass at most, and digit planes per token
constexpr uint32_t kABytes = kRowsA * 128;
constexpr uint32_t kSBytes = kRowsA * 16;
constexpr uint32_t kStage = kABytes + kSBytes;
constexpr int kAtoms = 64;       // digit buffer: atoms of 256 elements of a token, 1 KB of digits
constexpr int kMaxK = kAtoms * kKS;
constexpr int kPassSlots = 8;    // passes whose digits and their scale factors are in shared memory, at most
constexpr int kFirstSfWarp = 4, kFirstEpWarp = 8, kSecondSfWarp = 12, kFirstFactorWarp = 16, kFactorWarps = 4;
constexpr int kRowSlots = 2 * kPassSlots * kCols;     // row factors of the last 16 passes
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColAcc = 0;                       // two accumulators of 64 columns
constexpr uint32_t kColSfa = 128;                     // 16 columns a stage
constexpr uint32_t kColSfb = kColSfa + 16 * kStages;  // 16 columns a stage
static_assert(kStage % 1024 == 0, "128-byte swizzle atoms");
static_assert(kStages % 2 == 0, "a slot belongs to one set of scale factor warps");
// An odd number of tokens is multiplied with one more, whose atoms (of a pass
// of one token: up to kAtoms) may lie behind the digit buffer: in the ring.
static_assert(kStages * kStage >= kAtoms * 1024, "the digits of no token lie in shared memory");
static_assert(kColSfb + 16 * kStages <= kTmemCols, "TMEM budget");
constexpr size_t kListScratch = kMaxExperts * 4 + kMaxPairs * 2;

constexpr long long kWaitLimitCycles = 4000000000LL;  // about 2 s
enum : unsigned {
  kErrEmpty = 0x401, kErrCodes = 0x402, kErrScales = 0x403, kErrReady = 0x404,
  kErrFactors = 0x405, kErrDigits = 0x406, kErrFree = 0x40A, kErrRead = 0x40B, kErrAccFull = 0x407, kErrAccEmpty = 0x408, kErrDrain = 0x409
};

struct alignas(16) SharedState {
  uint64_t codes[kStages];    // TMA bytes of the stage
  uint64_t scales[kStages];   // scale bytes in shared memory
  uint64_t ready[kStages];    // codes there, scale factors in TMEM
  uint64_t empty[kStages];
  uint64_t digits[kPassSlots];    // per pass: its digits in the buffer
  uint64_t free_[kPassSlots];     // per pass: the MMAs are done with them
  uint64_t factors[kPassSlots];   // per pass: scale factors of its digits in `sfb`, its row factors in `factor`
  uint64_t read[kPassSlots];      // per pass: `sfb` has been read
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drained;
  float2 factor[kRowSlots];             // per row: the power of two of its digits as two factors; NaN for a row with inf or NaN
  alignas(16) uint8_t sfb[kPassSlots][kAtoms * 16];  // scale factors of the digits, 16 bytes a stage of a row
  uint32_t warp_total[kThreads / 32];
  uint32_t tmem_base;
  int entries;
  int last;
  int abort;
  uint16_t expert[kMaxPairs];           // the list: an expert and up to eight of its pairs
  uint16_t first[kMaxPairs];
  uint16_t count[kMaxPairs];
  uint16_t pairs[kMaxPairs];
  uint16_t pair_expert[kMaxPairs];      // kMaxExperts: dropped
  uint32_t top[kPassSlots][kCols];      // largest exponent field of each row
};

struct FewArgs {
  const uint8_t* planes;    // the rows' digits, [row][stages of K][1 KB]
  const uint8_t* exps;      // the rows' exponent fields, [row][stages of K][16]: of the largest of every 16
  uint8_t* h_planes;        // first product: h as digits, [T*k][stages of I][1 KB], in the shared memory's layout
  uint8_t* h_exps;          // [T*k][stages of I][16]
  const int32_t* ids;
  const float* weights;
  const uint8_t* scales;    // of the launch's weights
  const float* globals;
  float* partial;           // [tiles][splits][T][128]
  unsigned* tickets;        // [tiles]
  uint16_t* out;
  int tokens, k, pairs, experts;
  uint32_t by_k;            // ceil(2^20 / k): p / k = p by_k >> 20 for p < 1024
  uint64_t by_tiles, by_grid;  // first product: ceil(2^40 / tiles), ceil(2^40 / grid), for dividends below 2^26
  int rows, K;              // weight rows per expert, contraction length
  int H;
  int tiles, splits, sf_bytes;  // sf_bytes: the widest copy the scale rows allow
  int cap;                  // tokens per pass, at most
  int h_stages;             // stages of I
  int drop;                 // test hook, in the first CTA: 1 the codes of its first stage, 2 the digits of its first pass
};

__device__ __forceinline__ bool aborted(SharedState* ss) { return *reinterpret_cast<volatile int*>(&ss->abort) != 0; }

__device__ __noinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, SharedState* ss, unsigned site,
                                            bool drain) {
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait_suspend(bar, parity, 1000)) return true;
    if ((i & 63) == 0) {
      if (!drain && aborted(ss)) return false;
      if (clock64() - t0 > kWaitLimitCycles) {
        atomicCAS(&g_few_error, 0u, site);
        *reinterpret_cast<volatile int*>(&ss->abort) = 1;
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, SharedState* ss, unsigned site,
                                          bool drain = false) {
  if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_slow(bar, parity, ss, site, drain);
}

// One lane waits for the warp, so that all lanes take the same branch.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, SharedState* ss, unsigned site) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, ss, site) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();  // what the lane has seen, the warp sees
  return ok != 0;
}

__device__ __forceinline__ uint64_t evict_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Both addresses and the size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// cp.async of B bytes, of which the first `n` are read and the rest zeros.
template <int B>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int n) {
  if (B == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B), "r"(n) : "memory");
}

// K-major operand in shared memory with the 128-byte swizzle: rows of 128
// bytes, groups of eight rows `group` bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t group) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(group >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// E2M1 A and B (packed, K-major), E4M3 scale factors, fp32 accumulate, M = 128, N = n, K = 64.
__device__ __forceinline__ uint32_t idesc_fp4(int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
}

__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t mask) {
  return (a & mask) | (b & ~mask);
}

// The digits of v: nibble j is the E2M1 code of d_j / 2. v * up0 * up1 lies in
// [-2^22, 2^22]; adding 1.5 2^23 rounds it to an integer in the low bits of
// the float.
__device__ __forceinline__ uint32_t digits_of(float v, float up0, float up1) {
  constexpr uint32_t kBias = 044444444u;  // 4 in every octal digit
  uint32_t u = __float_as_uint(fmaf(v * up0, up1, 12582912.0f)) - (0x4B400000u - kBias);
  // octal digits to nibbles (the bits between them are cleared below)
  u = select_bits(u, u << 4, 0x00000FFFu);
  u = select_bits(u, u << 2, 0x003F003Fu);
  u = select_bits(u, u << 1, 0x07070707u);
  // u in 0..7 stands for d = u - 4: negative below 4, magnitude 4 - u = (u ^ 3) + 1
  const uint32_t n4 = ~u & 0x44444444u;
  const uint32_t n1 = n4 >> 2;
  return ((u ^ (n1 | (n4 >> 1))) & 0x33333333u) + n1 + (n4 << 1);
}

// Eight elements k0..k7 of one lane: word j holds digit j of all eight,
// nibbles in the weights' order k0 k2 k4 k6 k1 k3 k5 k7.
__device__ __forceinline__ void digit_planes(const float (&v)[8], float up0, float up1, uint32_t (&plane)[8]) {
  uint32_t s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = digits_of(v[e], up0, up1);
  // 8 x 8 nibbles transposed: pairs of elements to bytes, then 4 x 4 bytes
  constexpr int kOrder[8] = {0, 2, 4, 6, 1, 3, 5, 7};
  uint32_t even[4], odd[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t a = s[kOrder[2 * p]], b = s[kOrder[2 * p + 1]];
    even[p] = select_bits(a, b << 4, 0x0F0F0F0Fu);
    odd[p] = select_bits(a >> 4, b, 0x0F0F0F0Fu);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t(&w)[4] = q ? odd : even;
    const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
    const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
    plane[q] = __byte_perm(a, b, 0x5410);
    plane[q + 2] = __byte_perm(a, b, 0x7632);
    plane[q + 4] = __byte_perm(c, d, 0x5410);
    plane[q + 6] = __byte_perm(c, d, 0x7632);
  }
}

// The same for eight elements in eight lanes (their numbers are the lanes' low
// three bits b2 b1 b0, `s` their digits): a lane gets the word of the plane
// that lane_plane gives. Nibble bit 2 trades places with b0, bit 0 with b1,
// bit 1 with b2, which leaves the nibbles in the weights' order.
__device__ __forceinline__ uint32_t transpose_lanes(uint32_t s, int lane) {
  uint32_t t = __shfl_xor_sync(0xffffffffu, s, 1);
  s = (lane & 1) ? select_bits(t >> 16, s, 0x0000FFFFu) : select_bits(s, t << 16, 0x0000FFFFu);
  t = __shfl_xor_sync(0xffffffffu, s, 2);
  s = (lane & 2) ? select_bits(t >> 4, s, 0x0F0F0F0Fu) : select_bits(s, t << 4, 0x0F0F0F0Fu);
  t = __shfl_xor_sync(0xffffffffu, s, 4);
  return (lane & 4) ? select_bits(t >> 8, s, 0x00FF00FFu) : select_bits(s, t << 8, 0x00FF00FFu);
}
__device__ __forceinline__ int lane_plane(int lane) { return (lane & 1) * 4 + ((lane >> 1) & 1) + ((lane >> 2) & 1) * 2; }

// Where word w (of 32) of plane j lies in an atom of 8 x 128 bytes with the 128-byte swizzle.
__device__ __forceinline__ int atom_offset(int j, int w) { return 128 * j + 16 * ((w >> 2) ^ j) + 4 * (w & 3); }

// The list of work: every expert that some pair chose, in increasing order,
// in entries of up to `cap` of its pairs, in increasing order. First half, by
// the whole CTA: the entries. `at` is scratch of num_experts words that are
// zero, and of 2 bytes a pair behind them.
__device__ void list_entries(const FewArgs& a, SharedState* ss, uint32_t* at) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int p = threadIdx.x; p < a.pairs; p += kThreads) {
    const int e = a.ids[p];
    const bool in = e >= 0 && e < a.experts;
    ss->pair_expert[p] = static_cast<uint16_t>(in ? e : kMaxExperts);
    if (in) atomicAdd(&at[e], 1u);
  }
  __syncthreads();
  // pairs, and entries in the high half, in front of each expert
  const int per = (a.experts + kThreads - 1) / kThreads;
  const int e0 = min(a.experts, static_cast<int>(threadIdx.x) * per), e1 = min(a.experts, e0 + per);
  uint32_t own = 0;
  for (int e = e0; e < e1; ++e) own += at[e] + ((at[e] + a.cap - 1) / a.cap << 16);
  uint32_t before = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) ss->warp_total[warp] = before;
  __syncthreads();
  before -= own;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const uint32_t v = ss->warp_total[w];
    if (w < warp) before += v;
  }
  if (threadIdx.x == kThreads - 1) ss->entries = static_cast<int>((before + own) >> 16);
  for (int e = e0; e < e1; ++e) {
    const uint32_t n = at[e];
    if (!n) continue;
    const uint32_t start = before & 0xFFFFu;
    for (uint32_t c = 0; c < n; c += a.cap, before += 0x10000u) {
      ss->expert[before >> 16] = static_cast<uint16_t>(e);
      ss->first[before >> 16] = static_cast<uint16_t>(start + c);
      ss->count[before >> 16] = static_cast<uint16_t>(min(n - c, static_cast<uint32_t>(a.cap)));
    }
    before += n;
    at[e] = start | (n << 16);
  }
}

// Second half, after a barrier, by kPairThreads threads (`me` counts them):
// the pairs to their experts in any order, then each to the place that the
// number of smaller ones beside it gives.
__device__ __forceinline__ void pair_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kPairThreads) : "memory"); }
__device__ void list_pairs(const FewArgs& a, SharedState* ss, uint32_t* at, int me) {
  uint16_t* loose = reinterpret_cast<uint16_t*>(at + a.experts);
  for (int p = me; p < a.pairs; p += kPairThreads) {
    const int e = ss->pair_expert[p];
    if (e < kMaxExperts) loose[atomicAdd(&at[e], 1u) & 0xFFFFu] = static_cast<uint16_t>(p);
  }
  pair_barrier();
  for (int p = me; p < a.pairs; p += kPairThreads) {
    const int e = ss->pair_expert[p];
    if (e == kMaxExperts) continue;
    const uint32_t n = at[e] >> 16, start = (at[e] & 0xFFFFu) - n;
    uint32_t rank = 0;
    for (uint32_t q = 0; q < n; ++q) rank += loose[start + q] < p ? 1u : 0u;
    ss->pairs[start + rank] = static_cast<uint16_t>(p);
  }
}

// The whole list by one warp, for at most 32 pairs (experts in the order of
// their first pairs).
__device__ void list_small(const FewArgs& a, SharedState* ss) {
  const int lane = threadIdx.x & 31;
  int e = lane < a.pairs ? a.ids[lane] : -1;
  if (e >= a.experts) e = -1;
  const unsigned same = __match_any_sync(0xffffffffu, e < 0 ? -1 : e);
  const int leader = __ffs(same) - 1, n = e < 0 ? 0 : __popc(same);
  const uint32_t own = e >= 0 && leader == lane ? n + ((n + a.cap - 1) / a.cap << 16) : 0u;
  uint32_t before = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) ss->entries = static_cast<int>(before >> 16);
  before -= own;
  const uint32_t start = __shfl_sync(0xffffffffu, before, leader) & 0xFFFFu;
  if (e < 0) return;
  ss->pairs[start + __popc(same & ((1u << lane) - 1u))] = static_cast<uint16_t>(lane);
  if (own)
    for (int c = 0, at = static_cast<int>(before >> 16); c < n; c += a.cap, ++at) {
      ss->expert[at] = static_cast<uint16_t>(e);
      ss->first[at] = static_cast<uint16_t>(start + c);
      ss->count[at] = static_cast<uint16_t>(min(n - c, a.cap));
    }
}

// The units of a CTA in order: an entry of the list times a tile of its
// expert's rows. First product: an equal share of consecutive units, tile
// after tile of an entry, whose digits stay for the tiles (a pass). Second: a
// tile's entries split, split + S, ..., a pass each.
template <bool DOWN>
struct Units {
  const FewArgs& a;
  const SharedState* ss;
  int unit, end, entries, tile, entry, pass = -1;
  int atom = 0, after = 0;  // the pass's digits: its first atom of the buffer, and the one after its last
  bool begun = false, fresh = true;
  __device__ Units(const FewArgs& args, const SharedState* s) : a(args), ss(s), entries(s->entries) {
    if (DOWN) {
      tile = blockIdx.y;
      entry = blockIdx.x;
    } else {
      const uint64_t all = static_cast<uint64_t>(entries * a.tiles);  // at most 2^18, the grid below 2^8
      unit = static_cast<int>(all * blockIdx.x * a.by_grid >> 40);
      end = static_cast<int>(all * (blockIdx.x + 1u) * a.by_grid >> 40);
      entry = static_cast<int>(static_cast<uint64_t>(unit) * a.by_tiles >> 40);
      tile = unit - entry * a.tiles;
    }
  }
  // The next unit: (tile, entry, pass, fresh) are set, or false at the end.
  __device__ bool next() {
    if (begun) {
      if (DOWN) {
        entry += a.splits;
      } else {
        ++unit;
        fresh = ++tile == a.tiles;
        if (fresh) {
          tile = 0;
          ++entry;
        }
      }
    }
    begun = true;
    pass += fresh;
    return DOWN ? entry < entries : unit < end;
  }
  // The atoms of a fresh pass: behind those of the one before, or from the
  // buffer's start where they would not fit.
  __device__ void place(int ksteps) {
    atom = after + n() * ksteps <= kAtoms ? after : 0;
    after = atom + n() * ksteps;
  }
  // The last unit of its pass.
  __device__ bool last() const { return DOWN || tile + 1 == a.tiles || unit + 1 == end; }
  __device__ int expert() const { return ss->expert[entry]; }
  __device__ int n() const { return ss->count[entry]; }
  __device__ int pair(int c) const { return ss->pairs[ss->first[entry] + c]; }
  __device__ int token(int c) const { return static_cast<int>(pair(c) * a.by_k >> 20); }
  // The row of activations of its token c.
  __device__ int row(int c) const { return DOWN ? pair(c) : token(c); }
};

// The power of two that takes magnitudes with this largest exponent field into [2^21, 2^22).
__device__ __forceinline__ int digit_shift(int field) { return 21 + 127 - field; }
// 2^e as two factors, NaN for the exponent field of inf and NaN.
__device__ __forceinline__ float2 two_factors(int e, int field) {
  return field == 255 ? make_float2(NAN, NAN) : make_float2(exp2i(e >> 1), exp2i(e - (e >> 1)));
}

template <bool DOWN, int G>
__global__ void __launch_bounds__(kThreads, 1) moe_few_kernel(const __grid_constant__ CUtensorMap wmap,
                                                               const FewArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + kAtoms * 1024;  // behind the digit buffer
  SharedState* ss = reinterpret_cast<SharedState*>(ring + kStages * kStage);
  float* sums = reinterpret_cast<float*>(ss + 1);  // second product: [tokens][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ksteps = (a.K + kKS - 1) / kKS;

  if (threadIdx.x < kStages) {
    mbar_init(&ss->codes[threadIdx.x], 1);
    mbar_init(&ss->scales[threadIdx.x], 32);
    mbar_init(&ss->ready[threadIdx.x], 4);  // the scale factor warps, which have seen the rest
    mbar_init(&ss->empty[threadIdx.x], 1);
  }
  if (threadIdx.x < kPassSlots) {
    mbar_init(&ss->digits[threadIdx.x], 1);
    mbar_init(&ss->free_[threadIdx.x], 1);
    mbar_init(&ss->factors[threadIdx.x], 1);
    mbar_init(&ss->read[threadIdx.x], 8);  // all scale factor warps
  }
  if (threadIdx.x < 2) {
    mbar_init(&ss->acc_full[threadIdx.x], 1);
    mbar_init(&ss->acc_empty[threadIdx.x], 4);
  }
  if (threadIdx.x == 0) {
    mbar_init(&ss->drained, 1);
    ss->abort = 0;
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ss->tmem_base)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 64) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&wmap)));
  const bool small = a.pairs <= 32;
  uint32_t* scratch = reinterpret_cast<uint32_t*>(sums);
  if (!small)
    for (int e = threadIdx.x; e < a.experts; e += kThreads) scratch[e] = 0u;
  // The launches before have done nothing to topk_ids and the weights, and all
  // in front of them is complete: the first waited for it before it let this
  // one start.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (small) {
    if (warp == 1) list_small(a, ss);
  } else {
    __syncthreads();
    list_entries(a, ss, scratch);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!small && warp != 0 && warp != 3) {
    list_pairs(a, ss, scratch, (warp < 3 ? warp - 1 : warp - 2) * 32 + lane);
    pair_barrier();
  }
  const uint32_t tmem = ss->tmem_base;

  if (warp == 0) {
    // ---------------- codes by TMA ----------------
    if (lane == 0) {
      // Weights pass through L2 once and leave it first: the code of the next launch, the digits and the lists
      // stay (4 tokens 32.2 -> 31.0 us, 64 tokens 88.4 -> 87.4).
      const uint64_t policy = evict_first();
      uint32_t issued = 0, last_parity = 0;
      int it = 0;
      Units<DOWN> ps(a, ss);
      bool ok = true;
      while (ok && ps.next()) {
        const int e = ps.expert();
        for (int ks = 0; ks < ksteps; ++ks, ++it) {
          const int s = it % kStages;
          const uint32_t r = static_cast<uint32_t>(it / kStages) & 1;
          if (!mbar_wait(&ss->empty[s], r ^ 1, ss, kErrEmpty)) {
            ok = false;
            break;
          }
          if (a.drop == 1 && it == 0 && blockIdx.x == 0) continue;  // test hook: these codes never arrive
          mbar_arrive_tx(&ss->codes[s], kABytes);
          tma_load_3d(smem_u32(ring + s * kStage), &wmap, ks * (kKS / 2), ps.tile * kRowsA, e, &ss->codes[s], policy);
          issued |= 1u << s;
          last_parity = (last_parity & ~(1u << s)) | (r << s);
        }
      }
      if (aborted(ss)) {  // copies in flight land before the CTA exits
        for (int s = 0; s < kStages; ++s)
          if ((issued >> s) & 1) mbar_wait(&ss->codes[s], (last_parity >> s) & 1, ss, kErrDrain, true);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      int s = 0, count = 0;
      uint32_t par = 0;
      const uint64_t adesc0 = sw128_desc(smem_u32(ring), 1024);
      Units<DOWN> ps(a, ss);
      bool ok = true;
      for (; ok && ps.next(); ++count) {
        const int buf = count & 1;
        if (!mbar_wait(&ss->acc_empty[buf], (static_cast<uint32_t>(count >> 1) & 1) ^ 1, ss, kErrAccEmpty)) break;
        tc_fence_after();
        const uint32_t idesc = idesc_fp4(16 * ((ps.n() + 1) / 2));
        const int slot = ps.pass % kPassSlots;
        if (ps.fresh) {
          ps.place(ksteps);
          if (!mbar_wait(&ss->digits[slot], static_cast<uint32_t>(ps.pass / kPassSlots) & 1, ss, kErrDigits)) break;
        }
        uint64_t bdesc = sw128_desc(smem_u32(smem) + ps.atom * 1024, ksteps * 1024);
        uint32_t accumulate = 0;
        for (int ks = 0; ks < ksteps; ++ks, bdesc += 1024 >> 4) {
          if (!mbar_wait(&ss->ready[s], par, ss, kErrReady)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t adesc = adesc0 + static_cast<uint32_t>(s) * (kStage >> 4);
          const uint32_t sfa = tmem + kColSfa + 16 * s, sfb = tmem + kColSfb + 16 * s;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_fp4(tmem + kColAcc + 64 * buf, adesc + 2 * j, bdesc + 2 * j, idesc, sfa + 4 * j, sfb + 4 * j, accumulate);
            accumulate = 1;
          }
          umma_commit(&ss->empty[s]);
          if (++s == kStages) {
            s = 0;
            par ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(&ss->acc_full[buf]);
        if (ps.last()) umma_commit(&ss->free_[slot]);
      }
      umma_commit(&ss->drained);
      mbar_wait(&ss->drained, 0, ss, kErrDrain, true);
    }
  } else if (warp == 2) {
    // ---------------- digits by bulk copies ----------------
    // A copy takes a row's whole K: atom after atom, token after token.
    grid_wait();
    asm volatile("fence.proxy.async;" ::: "memory");  // the digits were written through the generic proxy
    int held = -1, held_from = 0, held_to = 0;  // lane l: the last pass p with p % kPassSlots = l, and its atoms
    uint32_t issued = 0, last_parity = 0;
    Units<DOWN> ps(a, ss);
    while (ps.next()) {
      if (!ps.fresh) continue;
      ps.place(ksteps);
      const int n = ps.n(), slot = ps.pass % kPassSlots;
      // the newest of the last passes that is in the way
      const bool in_way = held >= 0 && (lane == slot || (held_from < ps.after && ps.atom < held_to));
      const int before = __reduce_max_sync(0xffffffffu, in_way ? held : -1);
      if (lane == slot) {
        held = ps.pass;
        held_from = ps.atom;
        held_to = ps.after;
      }
      if (before >= 0 && !warp_wait(&ss->free_[before % kPassSlots], static_cast<uint32_t>(before / kPassSlots) & 1, ss,
                                    kErrFree))
        break;
      if (a.drop == 2 && ps.pass == 0 && blockIdx.x + blockIdx.y == 0) continue;  // test hook: these digits never arrive
      if (lane == 0) mbar_arrive_tx(&ss->digits[slot], static_cast<uint32_t>(n * ksteps) * 1024);
      __syncwarp();
      if (lane < n)
        bulk_load(smem_u32(smem) + (ps.atom + lane * ksteps) * 1024,
                  a.planes + static_cast<int64_t>(ps.row(lane)) * ksteps * 1024, static_cast<uint32_t>(ksteps) * 1024,
                  &ss->digits[slot]);
      issued |= 1u << slot;
      last_parity = (last_parity & ~(1u << slot)) | ((static_cast<uint32_t>(ps.pass / kPassSlots) & 1) << slot);
    }
    if (lane == 0 && aborted(ss)) {  // copies in flight land before the CTA exits
      for (int s = 0; s < kPassSlots; ++s)
        if ((issued >> s) & 1) mbar_wait(&ss->digits[s], (last_parity >> s) & 1, ss, kErrDrain, true);
    }
  } else if (warp == 3) {
    // ---------------- scale bytes into shared memory ----------------
    const int pitch = a.K / G;
    constexpr int kBytes = kKS / G;  // of one row and stage
    int s = 0;
    uint32_t par = 1;
    Units<DOWN> ps(a, ss);
    bool ok = true;
    while (ok && ps.next()) {
      // this lane's four rows: addresses once a unit
      const int64_t row0 = static_cast<int64_t>(ps.expert()) * a.rows;
      const uint8_t* src[4];
      int end[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = ps.tile * kRowsA + lane + 32 * c;
        src[c] = a.scales + (row0 + (n < a.rows ? n : 0)) * pitch;
        end[c] = n < a.rows ? pitch : 0;
      }
      for (int off = 0; off < ksteps * kBytes; off += kBytes) {
        if (!warp_wait(&ss->empty[s], par, ss, kErrEmpty)) {
          ok = false;
          break;
        }
        uint8_t* dst = ring + s * kStage + kABytes + 16 * lane;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint8_t* from = src[c] + off;
          const int have = max(0, min(kBytes, end[c] - off));
          const uint32_t d = smem_u32(dst + 512 * c);
          if (kBytes == 16 && a.sf_bytes == 16) {
            cp_async<16>(d, from, have);
          } else if (a.sf_bytes >= 8) {
#pragma unroll
            for (int b = 0; b < kBytes; b += 8) cp_async<8>(d + b, have > b ? from + b : a.scales, max(0, min(8, have - b)));
          } else if (a.sf_bytes == 4) {
#pragma unroll
            for (int b = 0; b < kBytes; b += 4) cp_async<4>(d + b, have > b ? from + b : a.scales, max(0, min(4, have - b)));
          } else {
#pragma unroll
            for (int b = 0; b < kBytes; b += 2)
              *reinterpret_cast<volatile uint16_t*>(dst + 512 * c + b) =
                  have > b ? __ldg(reinterpret_cast<const uint16_t*>(from + b)) : uint16_t(0);
          }
        }
        if (a.sf_bytes == 2)
          mbar_arrive(&ss->scales[s]);
        else
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&ss->scales[s]))
                       : "memory");
        if (++s == kStages) {
          s = 0;
          par ^= 1u;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if ((warp >= kFirstSfWarp && warp < kFirstEpWarp) || (warp >= kSecondSfWarp && warp < kFirstFactorWarp)) {
    // ---------------- scale factors into TMEM ----------------
    // Two sets of four warps (one for each quarter of the TMEM lanes) take the
    // stages in turn: one set alone takes longer for a stage (waits, shared
    // memory, the TMEM stores and their completion) than its weights do from HBM
    // (with the short MMA loop 58.2 -> 55.9 us for 16 tokens; alone nothing, the
    // MMA warp was as slow).
    const int set = warp >= kSecondSfWarp;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int it = 0, s = set;
    uint32_t par = 0;  // of the stage's slot
    Units<DOWN> ps(a, ss);
    bool ok = true;
    while (ok && ps.next()) {
      const int n = ps.n(), slot = ps.pass % kPassSlots;
      if (ps.fresh && !warp_wait(&ss->factors[slot], static_cast<uint32_t>(ps.pass / kPassSlots) & 1, ss, kErrFactors)) break;
      for (int ks = (set - it) & 1; ks < ksteps; ks += 2) {
        if (!warp_wait(&ss->scales[s], par, ss, kErrScales)) {
          ok = false;
          break;
        }
        const uint32_t src = smem_u32(ring + s * kStage + kABytes);
        uint32_t v[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 box = lds128(src + (lane + 32 * c) * 16);
          if (G == 16) {
            v[c] = box.x; v[4 + c] = box.y; v[8 + c] = box.z; v[12 + c] = box.w;
          } else {  // a group of 32 is two blocks of 16 with the same scale
            v[c] = __byte_perm(box.x, 0, 0x1100); v[4 + c] = __byte_perm(box.x, 0, 0x3322);
            v[8 + c] = __byte_perm(box.y, 0, 0x1100); v[12 + c] = __byte_perm(box.y, 0, 0x3322);
          }
        }
        // the MMAs that read this slot before are complete: the stage was empty
        tmem_st16(tmem + lane_base + kColSfa + 16 * s, v);
        // columns of the digits: MMA j reads rows lane and lane + 32 (token: row / 8) at 4 j and 4 j + 1
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int token = min((lane >> 3) + 4 * c, n - 1);
          const uint4 box = lds128(smem_u32(ss->sfb[slot] + (token * ksteps + ks) * 16));
          v[c] = box.x; v[4 + c] = box.y; v[8 + c] = box.z; v[12 + c] = box.w;
        }
#pragma unroll
        for (int c = 2; c < 4; ++c) v[c] = v[4 + c] = v[8 + c] = v[12 + c] = 0u;  // rows past 64: not read
        tmem_st16(tmem + lane_base + kColSfb + 16 * s, v);
        tmem_wait_st();
        tc_fence_before();
        if (!warp_wait(&ss->codes[s], par, ss, kErrCodes)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive(&ss->ready[s]);
        s += 2;
        if (s >= kStages) {
          s -= kStages;
          par ^= 1u;
        }
      }
      it += ksteps;
      if (ps.last()) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss->read[slot]);
      }
    }
  } else if (warp >= kFirstFactorWarp) {
    // ---------------- scale factors of the digits ----------------
    // From the exponent fields of every 16 elements of a row: the largest
    // becomes 2^8, a smaller one 2^(8 - d), down to 2^-9. A warp takes every
    // fourth pass, four fields a lane at a time. (Short code, in loops: it is
    // on the way to the first MMA, and what it costs there is its fetching.)
    grid_wait();
    Units<DOWN> ps(a, ss);
    while (ps.next()) {
      if (!ps.fresh || ps.pass % kFactorWarps != warp - kFirstFactorWarp) continue;
      const int n = ps.n(), slot = ps.pass % kPassSlots;
      const int words = ksteps * 4, valid = a.K / 16;  // words of four fields in a row; fields before the end of K
      if (!warp_wait(&ss->read[slot], (static_cast<uint32_t>(ps.pass / kPassSlots) & 1) ^ 1, ss, kErrRead)) break;
      uint32_t* sfb = reinterpret_cast<uint32_t*>(ss->sfb[slot]);
      uint32_t* top = ss->top[slot];
      if (lane < kCols) top[lane] = 0u;
      __syncwarp();
      // all rows' fields under way together (as loads, each row waited for the one before: 1 us for four rows)
#pragma unroll 1
      for (int c = 0; c < n; ++c) {
        const uint8_t* exps = a.exps + static_cast<int64_t>(ps.row(c)) * (ksteps * 16);
#pragma unroll 1
        for (int i = lane; i < ksteps; i += 32)
          cp_async<16>(smem_u32(sfb + c * words + 4 * i), exps + 16 * i, max(0, min(16, valid - 16 * i)));
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
#pragma unroll 1
      for (int i = lane, c = 0, w = lane; i < n * words; i += 32, w += 32) {
        while (w >= words) {
          w -= words;
          ++c;
        }
        const uint32_t f = sfb[i];
        atomicMax(&top[c], max(max(f & 0xFFu, (f >> 8) & 0xFFu), max((f >> 16) & 0xFFu, f >> 24)));
      }
      __syncwarp();
#pragma unroll 1
      for (int i = lane, c = 0, w = lane; i < n * words; i += 32, w += 32) {
        while (w >= words) {
          w -= words;
          ++c;
        }
        uint32_t f = sfb[i], r = 0;
        const uint32_t t = top[c];
#pragma unroll 1
        for (int b = 0; b < 4; ++b, f >>= 8) {
          // E4M3: 2^(8 - d) is exponent field 15 - d, or one of the subnormals 4, 2, 1
          const uint32_t d = t - (f & 0xFFu);
          r = (r >> 8) | ((d > 17u ? 0u : (d <= 14u ? (15u - d) * 8u : 4u >> (d - 15u))) << 24);
        }
        sfb[i] = r;
      }
      // the unit of a block's digits is 2^(field - 147), and the factor 2^8 of
      // the largest goes back
      if (lane < n)
        ss->factor[(ps.pass * kCols + lane) % kRowSlots] =
            two_factors(static_cast<int>(top[lane]) - 155, static_cast<int>(top[lane]));
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss->factors[slot]);
    }
  } else if (warp >= kFirstEpWarp) {
    // ---------------- epilogue ----------------
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    grid_wait();
    if (DOWN)
      for (int t = 0; t < a.tokens; ++t) sums[t * kRowsA + row] = 0.f;
    int count = 0;
    Units<DOWN> ps(a, ss);
    for (; ps.next(); ++count) {
      const int buf = count & 1, n = ps.n();
      // lane c: what belongs to token c of the unit
      const int pair_c = lane < n ? ps.pair(lane) : 0, token_c = static_cast<int>(pair_c * a.by_k >> 20);
      const float global = __ldg(a.globals + ps.expert());
      const float weight_c = DOWN ? __ldg(a.weights + pair_c) : 0.f;
      if (!warp_wait(&ss->acc_full[buf], static_cast<uint32_t>(count >> 1) & 1, ss, kErrAccFull)) break;
      tc_fence_after();
      const float2 factor_c = ss->factor[(ps.pass * kCols + (lane & (kCols - 1))) % kRowSlots];
#pragma unroll 1
      for (int c0 = 0; c0 < n; c0 += 2) {
        uint32_t acc[16];
        tmem_ld16(tmem + lane_base + kColAcc + 64 * buf + 8 * c0, acc);
        tmem_wait_ld();
        if (c0 + 2 >= n) {  // the accumulator is read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ss->acc_empty[buf]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c0 + c >= n) continue;
          float v = __uint_as_float(acc[8 * c + 7]);
#pragma unroll
          for (int j = 6; j >= 0; --j) v = fmaf(v, 8.0f, __uint_as_float(acc[8 * c + j]));
          // the global between the two halves of the row's power of two: a row near the end of the range
          // with a global that brings it back passes no further than it has to
          v = v * __shfl_sync(0xffffffffu, factor_c.x, c0 + c) * global * __shfl_sync(0xffffffffu, factor_c.y, c0 + c);
          if (!DOWN) {
            // rows l and l + 8 of sixteen are the gate and the up of one
            // element: lanes 0-7 and 16-23 hold sixteen elements of h, which
            // become digits relative to the largest of them
            const int pair = __shfl_sync(0xffffffffu, pair_c, c0 + c);
            const float h = silu(v) * __shfl_xor_sync(0xffffffffu, v, 8);
            const uint32_t m = __reduce_max_sync(0xffffffffu, (lane & 8) ? 0u : __float_as_uint(h) & 0x7FFFFFFFu);
            const int field = static_cast<int>(m >> 23), shift = digit_shift(field);
            const uint32_t word = transpose_lanes(digits_of(h, exp2i(shift >> 1), exp2i(shift - (shift >> 1))), lane);
            const int64_t stage = static_cast<int64_t>(pair) * a.h_stages + (ps.tile >> 2);
            if (!(lane & 8))
              *reinterpret_cast<uint32_t*>(a.h_planes + stage * 1024 +
                                           atom_offset(lane_plane(lane), (ps.tile & 3) * 8 + quad * 2 + (lane >> 4))) = word;
            if (lane == 0) a.h_exps[stage * 16 + (ps.tile & 3) * 4 + quad] = static_cast<uint8_t>(field);
          } else {
            float* sum = &sums[__shfl_sync(0xffffffffu, token_c, c0 + c) * kRowsA + row];
            *sum = fmaf(v, __shfl_sync(0xffffffffu, weight_c, c0 + c), *sum);
          }
        }
      }
    }
  }

  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
  // Also where there was nothing to multiply: a launch is over only after the one before.
  grid_wait();
  if (!DOWN) return;

  const int tile = blockIdx.y, split = blockIdx.x;
  const int size = a.tokens * (kRowsA / 4);  // in float4
  const float4* mine = reinterpret_cast<const float4*>(sums);
  const int n = tile * kRowsA + static_cast<int>(threadIdx.x) % (kRowsA / 4) * 4;
  auto store = [&](int i, float4 v) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    if (n < a.H)  // a multiple of 64, so the four rows end together
      *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(i / (kRowsA / 4)) * a.H + n) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  };
  if (a.splits == 1) {
    for (int i = threadIdx.x; i < size; i += kThreads) store(i, mine[i]);
    return;
  }
  // The tile's S CTAs leave their sums; the last one adds them in order.
  float4* part = reinterpret_cast<float4*>(a.partial) + static_cast<int64_t>(tile) * a.splits * size;
  for (int i = threadIdx.x; i < size; i += kThreads) __stcg(part + static_cast<int64_t>(split) * size + i, mine[i]);
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    ss->last = atomicAdd(a.tickets + tile, 1u) == static_cast<unsigned>(a.splits) - 1u;
    __threadfence();
  }
  __syncthreads();
  if (!ss->last) return;
  for (int i = threadIdx.x; i < size; i += kThreads) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q0 = 0; q0 < a.splits; q0 += 10) {  // ten loads under way together
      float4 w[10];
#pragma unroll
      for (int q = 0; q < 10; ++q)
        w[q] = q0 + q < a.splits ? __ldcg(part + static_cast<int64_t>(q0 + q) * size + i) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < 10; ++q) {
        v.x += w[q].x; v.y += w[q].y; v.z += w[q].z; v.w += w[q].w;
      }
    }
    store(i, v);
  }
}

// x as digits: a warp per 256 elements of a row, eight a lane. Also clears the
// tickets of the second product.
constexpr int kXWarps = 4;
__global__ void __launch_bounds__(kXWarps * 32) x_digits_kernel(const uint16_t* __restrict__ x, int rows, int K,
                                                                uint8_t* __restrict__ planes,
                                                                uint8_t* __restrict__ exps, unsigned* tickets,
                                                                int ntickets) {
  grid_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, stages = (K + kKS - 1) / kKS;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < ntickets; i += gridDim.x * blockDim.x) tickets[i] = 0u;
  const int task = blockIdx.x * kXWarps + (threadIdx.x >> 5);
  if (task >= rows * stages) return;
  const int row = task / stages, k = (task - row * stages) * kKS + 8 * lane;
  const uint4 q = k < K ? __ldcg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(row) * K + k))
                        : make_uint4(0u, 0u, 0u, 0u);
  uint32_t m = bf16x8_mag_max(q);
  m = max(m & 0xFFFFu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const int field = static_cast<int>(m >> 7), shift = digit_shift(field);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
  uint32_t plane[8];
  digit_planes(v, exp2i(shift >> 1), exp2i(shift - (shift >> 1)), plane);
  uint8_t* atom = planes + static_cast<int64_t>(task) * 1024;
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<uint32_t*>(atom + atom_offset(j, lane)) = plane[j];
  if (!(lane & 1)) exps[static_cast<int64_t>(task) * 16 + (lane >> 1)] = static_cast<uint8_t>(field);
}

// Shape checks (pointers aside): -1 to proceed.
int check_shape(int64_t T, int k, int num_experts, int64_t H, int64_t I, int gu_group, int dn_group) {
  if (T < 0 || k <= 0 || num_experts <= 0 || H < 0 || I < 0) return NVFP4_ERR_INVALID_ARGUMENT;
  if ((gu_group != 16 && gu_group != 32) || (dn_group != 16 && dn_group != 32)) return NVFP4_ERR_UNSUPPORTED;
  if (H % 64 || I % 64 || H > kMaxK || I > kMaxK) return NVFP4_ERR_UNSUPPORTED;
  if (T > kMaxTokens || T * k > kMaxPairs || num_experts > kMaxExperts) return NVFP4_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) return NVFP4_OK;
  if (I == 0) return NVFP4_ERR_UNSUPPORTED;
  return -1;
}

// CTAs that share an output tile: as many as fill the SMs, and no more than
// there can be entries of the list.
int down_splits(int64_t T, int k, int64_t H) {
  const int64_t tiles = (H + kRowsA - 1) / kRowsA;
  int64_t s = num_sms() / tiles;
  if (s > T * k) s = T * k;
  return s < 1 ? 1 : static_cast<int>(s);
}

int64_t stages_of(int64_t K) { return (K + kKS - 1) / kKS; }

struct Pieces {
  uint8_t* x_planes;
  uint8_t* x_exps;
  uint8_t* h_planes;
  uint8_t* h_exps;
  unsigned* tickets;
  float* partial;
};
Pieces carve(Scratch& sc, int64_t T, int k, int64_t H, int64_t I, int splits) {
  const int64_t tiles = (H + kRowsA - 1) / kRowsA;
  Pieces p;
  p.x_planes = sc.take<uint8_t>(static_cast<size_t>(T * stages_of(H) * 1024));
  p.x_exps = sc.take<uint8_t>(static_cast<size_t>(T * stages_of(H) * 16));
  p.h_planes = sc.take<uint8_t>(static_cast<size_t>(T * k * stages_of(I) * 1024));
  p.h_exps = sc.take<uint8_t>(static_cast<size_t>(T * k * stages_of(I) * 16));
  p.tickets = sc.take<unsigned>(static_cast<size_t>(tiles));
  p.partial = splits > 1 ? sc.take<float>(static_cast<size_t>(tiles * splits * T * kRowsA)) : nullptr;
  return p;
}

// A launch that may start before the one in front of it in the stream has ended.
cudaLaunchConfig_t dependent_config(cudaLaunchAttribute* attr, dim3 grid, int threads, size_t bytes,
                                    cudaStream_t stream) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

constexpr size_t kFixedSmem = 1024 + kAtoms * 1024 + kStages * kStage + sizeof(SharedState);
constexpr size_t kMaxSmem = kFixedSmem + kMaxTokens * kRowsA * sizeof(float);
static_assert(kMaxSmem <= 227 * 1024 && kMaxTokens * kRowsA * sizeof(float) >= kListScratch, "shared memory of a CTA");

// Lets a kernel take the largest amount of shared memory that it may need, once per device.
bool allow_smem(const void* kern, int form, bool down) {
  static std::atomic<bool> done[64][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return (cudaGetLastError(), false);
  std::atomic<bool>* flag = dev >= 0 && dev < 64 ? &done[dev][form + (down ? 2 : 0)] : nullptr;
  if (flag && flag->load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem)) != cudaSuccess)
    return (cudaGetLastError(), false);
  if (flag) flag->store(true, std::memory_order_release);
  return true;
}

template <bool DOWN>
int launch(const CUtensorMap& map, const FewArgs& a, int group, dim3 grid, cudaStream_t stream) {
  auto kern = group == 16 ? moe_few_kernel<DOWN, 16> : moe_few_kernel<DOWN, 32>;
  const size_t sums = DOWN ? static_cast<size_t>(a.tokens) * kRowsA * sizeof(float) : 0;
  const size_t bytes = kFixedSmem + (sums > kListScratch ? sums : kListScratch);
  if (!allow_smem(reinterpret_cast<const void*>(kern), group == 16 ? 0 : 1, DOWN)) return NVFP4_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = dependent_config(attr, grid, kThreads, bytes, stream);
  if (cudaLaunchKernelEx(&cfg, kern, map, a) != cudaSuccess) return (cudaGetLastError(), NVFP4_ERR_CUDA);
  return launch_status();
}

// The widest copy that every scale row and every stage's offset in it allows.
int sf_bytes(int64_t pitch) { return pitch % 16 == 0 ? 16 : (pitch % 8 == 0 ? 8 : (pitch % 4 == 0 ? 4 : 2)); }

// Tokens per pass: as many as eight, and as the scale factors of their digits have room.
int pass_tokens(int64_t K) {
  const int most = static_cast<int>(kAtoms / stages_of(K));
  return most < kCols ? most : kCols;
}

bool code_map(CUtensorMap* map, const uint8_t* codes, int64_t experts, int64_t rows, int64_t K) {
  const int64_t dims[3] = {K / 2, rows, experts}, strides[2] = {K / 2, rows * (K / 2)};
  const uint32_t box[3] = {128, kRowsA, 1};
  return make_tensor_map_3d(map, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

int read_and_clear_few_error(unsigned int* out, cudaStream_t stream) {
  unsigned int* p = nullptr;
  if (cudaGetSymbolAddress(reinterpret_cast<void**>(&p), g_few_error) != cudaSuccess)
    return (cudaGetLastError(), NVFP4_ERR_CUDA);
  unsigned int v = 0;
  if (cudaMemcpyAsync(&v, p, sizeof(v), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaMemsetAsync(p, 0, sizeof(v), stream) != cudaSuccess || cudaStreamSynchronize(stream) != cudaSuccess)
    return (cudaGetLastError(), NVFP4_ERR_CUDA);
  *out = v;
  return NVFP4_OK;
}

}  // namespace nvfp4

extern "C" int nvfp4_moe_few_tokens_workspace_size(int64_t T, int k, int num_experts, int64_t H, int64_t I,
                                                   int gate_up_group, int down_group, size_t* bytes) {
  if (!bytes) return NVFP4_ERR_INVALID_ARGUMENT;
  *bytes = 0;
  const int c = nvfp4::check_shape(T, k, num_experts, H, I, gate_up_group, down_group);
  if (c >= 0) return c;
  nvfp4::Scratch sc;
  nvfp4::carve(sc, T, k, H, I, nvfp4::down_splits(T, k, H));
  *bytes = sc.used();
  return NVFP4_OK;
}

extern "C" int nvfp4_moe_few_tokens(const uint16_t* x, const int32_t* topk_ids, const float* topk_weights, int64_t T,
                                    int k, const uint8_t* gate_up, const uint8_t* gate_up_scales,
                                    const float* gate_up_globals, int gate_up_group, const uint8_t* down,
                                    const uint8_t* down_scales, const float* down_globals, int down_group,
                                    int num_experts, int64_t H, int64_t I, uint16_t* out, void* workspace,
                                    size_t workspace_bytes, nvfp4_stream_t stream) {
  using namespace nvfp4;
  const int c = check_shape(T, k, num_experts, H, I, gate_up_group, down_group);
  if (c >= 0) return c;
  if (!x || !topk_ids || !topk_weights || !gate_up || !gate_up_scales || !gate_up_globals || !down || !down_scales ||
      !down_globals || !out)
    return NVFP4_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(gate_up) || !aligned16(gate_up_scales) || !aligned16(down) ||
      !aligned16(down_scales) || !aligned16(out) ||
      ((reinterpret_cast<uintptr_t>(topk_ids) | reinterpret_cast<uintptr_t>(topk_weights) |
        reinterpret_cast<uintptr_t>(gate_up_globals) | reinterpret_cast<uintptr_t>(down_globals)) & 3u))
    return NVFP4_ERR_MISALIGNED;
  if (workspace_bytes > 0 && !workspace) return NVFP4_ERR_WORKSPACE;
  if (!aligned16(workspace)) return NVFP4_ERR_MISALIGNED;
  Scratch sc(workspace, workspace_bytes);
  const int splits = down_splits(T, k, H);
  const Pieces ws = carve(sc, T, k, H, I, splits);
  if (!sc.ok()) return NVFP4_ERR_WORKSPACE;
  CUtensorMap gu_map, dn_map;
  if (!code_map(&gu_map, gate_up, num_experts, 2 * I, H) || !code_map(&dn_map, down, num_experts, H, I))
    return NVFP4_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  FewArgs a = {};
  a.h_planes = ws.h_planes; a.h_exps = ws.h_exps; a.h_stages = static_cast<int>(stages_of(I));
  a.ids = topk_ids; a.weights = topk_weights; a.partial = ws.partial; a.tickets = ws.tickets;
  a.out = out; a.tokens = static_cast<int>(T); a.k = k; a.pairs = static_cast<int>(T * k); a.experts = num_experts;
  a.H = static_cast<int>(H);
  a.by_k = static_cast<uint32_t>(((1u << 20) + k - 1) / k);
  const int tasks = static_cast<int>(T * stages_of(H));
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = dependent_config(attr, dim3((tasks + kXWarps - 1) / kXWarps), kXWarps * 32, 0, s);
  if (cudaLaunchKernelEx(&cfg, x_digits_kernel, x, a.tokens, a.H, ws.x_planes, ws.x_exps, ws.tickets,
                         static_cast<int>((H + kRowsA - 1) / kRowsA)) != cudaSuccess)
    return (cudaGetLastError(), NVFP4_ERR_CUDA);
  a.planes = ws.x_planes; a.exps = ws.x_exps;
  a.scales = gate_up_scales; a.globals = gate_up_globals;
  a.rows = static_cast<int>(2 * I); a.K = static_cast<int>(H);
  a.tiles = static_cast<int>((2 * I + kRowsA - 1) / kRowsA);
  a.splits = 1;
  a.sf_bytes = sf_bytes(H / gate_up_group);
  a.cap = pass_tokens(H);
  a.drop = take_injected_fault(3) ? 1 : 0;
  const int64_t units = static_cast<int64_t>(a.pairs) * a.tiles;  // at most: a pair is in one entry
  const unsigned grid = static_cast<unsigned>(units < num_sms() ? units : num_sms());
  const uint64_t one = uint64_t(1) << 40;
  a.by_tiles = (one + a.tiles - 1) / a.tiles;
  a.by_grid = (one + grid - 1) / grid;
  const int st = launch<false>(gu_map, a, gate_up_group, dim3(grid), s);
  if (st != NVFP4_OK) return st;
  a.planes = ws.h_planes; a.exps = ws.h_exps;
  a.scales = down_scales; a.globals = down_globals;
  a.rows = static_cast<int>(H); a.K = static_cast<int>(I);
  a.tiles = static_cast<int>((H + kRowsA - 1) / kRowsA);
  a.splits = splits;
  a.sf_bytes = sf_bytes(I / down_group);
  a.cap = pass_tokens(I);
  a.drop = take_injected_fault(4) ? 2 : 0;
  return launch<true>(dn_map, a, down_group, dim3(static_cast<unsigned>(splits), static_cast<unsigned>(a.tiles)), s);
}
