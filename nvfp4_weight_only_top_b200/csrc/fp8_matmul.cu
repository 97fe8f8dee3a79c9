// Products of E4M3 rows with E4M3 weights, both with f32 block scales, on the tensor cores:
//   out[m, n] = sum over blocks kb of 128 inputs of
//               a_scales[m, kb] * b_scales[e, n / 128, kb] * (sum over k in kb of a[m, k] b[e, n, k])
// for the rows m of expert e.
//
// A tile is up to 128 rows of one expert (the 128 TMEM lanes) times BN outputs, or with a pair of CTAs
// up to 256 rows.  Each block of 128 inputs is one pipeline stage (one 128-byte swizzle row of E4M3) and
// one group of four tcgen05.mma kind::f8f6f4 (K = 32) into one of kBufs f32 accumulators in TMEM; the
// epilogue warps take that accumulator to registers, multiply it with the block's scale and add it to
// the running sum there, while the tensor core works on the next blocks in the others.  With rows as
// lanes a thread's scale is one number per block (its row's times the weight tile's), so a block costs
// a thread one multiply-add per output.  The tensor cores' sums of 128 products are f32 (measured:
// within 1e-6 of the largest product).
//
//   warps 0-7  epilogue: warp w the lanes 32 (w % 4) .. +31 and the columns of half w / 4;
//   then       TMA of the rows and the weights: one warp of a pair's CTA, else two, a block each in turn (the waits
//              and the issue of one took a warp about 400 clocks, the time of a block where CTAs are few: 64 rows x
//              5120 x 5120 13.8 us, now 10.5);
//   then       two warps for the MMAs (of a pair: in CTA 0);
//   last       copies of the scales to shared memory.
//
// A pair (cta_group::2) shares the weights: each CTA loads half of the BN weight rows and its own 128
// rows, 32 KB a block instead of 48, which the L2 can deliver in the time of the MMAs (512 clocks).
//
// Measured: 65787 rows over 32 experts x 5120 x 5120.  A few calls: 1.61 ms, 2.14 PFLOP/s, 0.65 of twice the measured
// burst BF16 rate.  Six seconds of calls: 1.88 ms each at 990 W (the power cap) and 1380 MHz, 1.83 PFLOP/s, 0.67 of
// twice the sustained BF16 rate.  Without its multiply-adds the same kernel takes 1.3 ms in a few calls: they fill a
// quarter of the issue slots, and a wait for an accumulator, its loads and they are one chain a warp (tensor pipe busy
// 62 %, issue slots 65 %: neither is full).  Decode batches read the weights: 67 rows over 32 experts x 5120 x 5120
// with 19 of them live 87 us, 490 MB at 0.86 of the measured copy's rate.
//
// Few tiles of long rows are shared by a cluster of up to eight CTAs, each a run of the blocks: with one CTA a tile
// the chain of its blocks is the time (64 rows x 512 x 5120: 10.5 us, five CTAs a tile 6.8).  Each leaves its sums in
// its shared memory and adds up a part of the rows from all of them, in order.
//
// Rows of the tile behind the expert's last (the next expert's, or what the stage held before) and
// columns behind N fill lanes and columns that are not stored; TMA fills inputs behind K with zeros.
#define MOE_OWN_STATUS
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "per_device.h"
#include "tc_pair.cuh"

namespace moe {

namespace {

constexpr int kTileM = 128;             // rows of one CTA
constexpr int kABytes = kTileM * 128;
constexpr int kMmaWarps = 2;
constexpr int kMaxExperts = 1024;
constexpr int kSuper = 8;               // row tiles taken together over the output tiles (L2 reuse)
constexpr int kRing = 4;                // groups of four blocks' scales in shared memory
constexpr int kMaxParts = kFp8MaxParts;

template <int BN, bool PAIR>
struct Cfg {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kEpiWarps = 8;
  static constexpr int kTmaWarps = BN == 256 ? 1 : 2;
  static constexpr int kThreads = 32 * (kEpiWarps + kTmaWarps + kMmaWarps + 1);
  static constexpr int kBRows = BN / kCtas;              // weight rows a CTA loads
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStage;        // 8, 6, 6
  static constexpr int kBufs = 512 / BN;
  // BN = 256 leaves room for two accumulators only, too few to cover the way from a block's MMAs (512 clocks) over
  // the epilogue's loads back to the MMAs that reuse its accumulator if that were one chain: its columns are two
  // halves of 128, each a chain of its own.
  static constexpr int kSplit = BN == 256 ? 2 : 1;
  // Shared memory, from a 1024-byte boundary: stages, barriers, scales, outputs, tile counts.
  static constexpr int kFull = kStages * kStage;         // [kStages] barriers
  static constexpr int kEmpty = kFull + 8 * kStages;     // [kStages]
  static constexpr int kDFull = kEmpty + 8 * kStages;    // [kSplit][kBufs]
  static constexpr int kDEmpty = kDFull + 8 * kSplit * kBufs;   // [kSplit][kBufs]
  static constexpr int kSFull = kDEmpty + 8 * kSplit * kBufs;   // [kRing]
  static constexpr int kSEmpty = kSFull + 8 * kRing;     // [kRing]
  static constexpr int kTmem = kSEmpty + 8 * kRing;
  static constexpr int kScaleHalves = BN == 256 ? 2 : 1; // weight tiles (of 128 outputs) a tile spans
  static constexpr int kScaleSlot = kTileM * 16 + 32;
  static constexpr int kScales = kStages * kStage + 512; // [kRing] scales of four blocks: of 128 rows, of two halves
  static constexpr int kOut = kScales + kRing * kScaleSlot;   // [8] 2 KB: the epilogue warps' rows on their way out
  static constexpr int kPre = kOut + kEpiWarps * 2048;
  static constexpr int kSmem = kPre + (kMaxExperts + 1) * 4 + 1024;
  static_assert(kStages % kTmaWarps == 0 && kStages % kMmaWarps == 0 && kBufs % (kMmaWarps / kSplit) == 0, "turns");
  static_assert(kTmem + 4 <= kScales && kSmem <= 232448, "shared memory");
};

struct Maps {
  CUtensorMap a[3];                     // [M, K] bytes, boxes of 128 B x 32, 64, 128 rows, 128B swizzle
  CUtensorMap b;                        // [E N, K] bytes, boxes of 128 B x kBRows rows
};

// kind::f8f6f4 with E4M3 operands (format 0 of both in the instruction descriptor), f32 accumulator.
template <bool PAIR>
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// One multiply-add of a running sum.  (Two at a time, fma.f32x2, has the same rate and made the compiler move
// half of the loaded values into register pairs, half as many instructions again.)  Volatile: x comes from
// tcgen05.ld, and only the wait before it, which names no register, makes it valid.
__device__ __forceinline__ void fma_acc(float& acc, float x, float s) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(x), "f"(s));
}
// 16 consecutive 32-bit TMEM columns of this thread's lane, as f32.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}
// True in one lane, the same at every call.  The loops around it are run by the whole warp: the MMA's
// operands then are uniform values of a converged warp (with the loop inside `if (lane == 0)` the
// issue of a block's MMAs took 2.5 times as long).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's arrival on `bar` once its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Barriers by their shared-memory address (32 bits, where a pointer would cost the epilogue two registers).
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same without waiting at all: try_wait may suspend the thread for some microseconds, which a look ahead at
// a block that does not come (a tile's last) would pay for.
__device__ __forceinline__ bool bar_peek(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Gives up after kWaitCycles (looked at every 64 tests: a waiting warp should take few issue slots), records a
// timeout in g_status and returns false.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (bar_test(bar, parity)) return true;
    if (clock64() - t0 > kWaitCycles) {
      atomicExch(&g_status, kStatusTimeout);
      return false;
    }
  }
}
// A whole warp's wait; false in all lanes if it gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xFFFFFFFFu, bar_test(bar, parity))) return true;
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity));
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Arrival on a barrier of the pair's CTA 0 (cluster address), with the default release at CTA scope: what it
// orders is tensor memory, by the tcgen05 fence before it (a release at cluster scope waits for the
// thread's every earlier access, about 1500 clocks a block here).
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Arrives on `bar` (of a pair: in both CTAs) when the MMAs this thread issued so far complete.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The register split of a block with BN = 256, whose epilogue threads hold 128 running sums: it starts with 384 x
// 168 registers (checked by the launcher); the epilogue's 256 threads then take 216 each and the others keep
// 72: 64512 together.
constexpr int kRegsLaunch = 168, kRegsEpi = 216, kRegsRest = 72;
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// The end of a block: every thread of the CTA (of the cluster) in its own role's code.
template <bool CLUSTER, int THREADS>
__device__ __forceinline__ void all_done() {
  tc_fence_before();
  if (CLUSTER)
    cluster_sync();
  else
    named_bar_sync(0, THREADS);
  tc_fence_after();
}

// A TMA load counted on `bar`: a barrier of the pair's CTA 0 (cluster address), or this CTA's own.
template <bool PAIR>
__device__ __forceinline__ void tma_load_to(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Expert e's rows, taken into [0, M] so that no offset reaches outside the tensors.
__device__ __forceinline__ void expert_rows(const Fp8Matmul& p, int e, int64_t& lo, int64_t& hi) {
  if (!p.offsets) {
    lo = 0;
    hi = p.M;
    return;
  }
  lo = min(max((int64_t)__ldg(p.offsets + e), (int64_t)0), p.M);
  hi = min(max((int64_t)__ldg(p.offsets + e + 1), lo), p.M);
}

// Rows of the box that holds a CTA's rows: 32, 64 or 128 (each TMA instruction costs its issue), 0 for none.
__device__ __forceinline__ int box_of(int rows) { return rows > 64 ? 128 : rows > 32 ? 64 : rows > 0 ? 32 : 0; }

// Blocks of a part: a multiple of four, the scales' groups (only the last part may have fewer).
__host__ __device__ __forceinline__ int part_blocks(int kall, int parts) { return (kall + 4 * parts - 1) / (4 * parts) * 4; }

struct Tile {
  int e, rows, n0;                      // rows: of the tile, both CTAs' of a pair
  int row0;
};
// Tile tt of the list: expert by expert (pre[e]: row tiles of the experts before), kSuper row tiles
// over all output tiles at a time.
__device__ __forceinline__ Tile find_tile(const Fp8Matmul& p, const int* pre, int ntiles, int bn, int tile_m, int tt) {
  int e = 0, hi = p.E;
  while (hi - e > 1) {
    const int mid = (e + hi) >> 1;
    if ((int64_t)pre[mid] * ntiles <= tt)
      e = mid;
    else
      hi = mid;
  }
  const int l = tt - pre[e] * ntiles, mt = pre[e + 1] - pre[e];
  const int sup = l / (kSuper * ntiles), in = l - sup * kSuper * ntiles;
  const int h = min(kSuper, mt - sup * kSuper);
  const int n = in / h, m = sup * kSuper + in - n * h;
  int64_t lo, end;
  expert_rows(p, e, lo, end);
  Tile t;
  t.e = e;
  t.n0 = n * bn;
  t.row0 = (int)lo + m * tile_m;
  t.rows = (int)min((int64_t)tile_m, end - t.row0);
  return t;
}

// A warp's 32 rows of N running sums to row-major memory, `rows` of them, through 2 KB of shared memory: a
// round takes 64 bytes of every row, each lane its own row in (chunk c of row r at c ^ (r / 2) % 4, free of
// bank conflicts both ways) and then 16 bytes of eight rows at a time out.  Stored straight from the lanes, a
// 16-byte store would touch 32 rows, and the stores of a tile took as long as eight blocks of inputs.
// column(c): the tile's column of sum c; n: outputs from the tile's first column on.
template <int N, bool F32, typename Column>
__device__ __forceinline__ void store_rows(const float (&acc)[N], uint32_t stage, uint8_t* row0, int64_t pitch,
                                           int rows, int n, int lane, Column column) {
  constexpr int kPer = F32 ? 16 : 32;                   // columns of a round
  const uint32_t mine = stage + lane * 64, swz = (lane >> 1) & 3;
#pragma unroll
  for (int c = 0; c < N; c += kPer) {
    __syncwarp();                                       // the round before has been read
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (F32)
          w[j] = __float_as_uint(acc[c + 4 * i + j]);
        else
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(acc[c + 8 * i + 2 * j + 1]), "f"(acc[c + 8 * i + 2 * j]));
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((i ^ swz) << 4)), "r"(w[0]), "r"(w[1]),
                   "r"(w[2]), "r"(w[3])
                   : "memory");
    }
    __syncwarp();
    const int col = column(c) + (lane & 3) * (kPer / 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)));
      if (r < rows && col < n) *reinterpret_cast<uint4*>(row0 + r * pitch + (int64_t)col * (F32 ? 4 : 2)) = v;
    }
  }
}

// The sums of a tile's parts, in order, by the CTA `part` of a cluster for its share of the rows: every CTA's are
// [128][BN + 4] f32 from `sm` on.
template <int BN>
__device__ __forceinline__ void sum_parts(const Fp8Matmul& p, const Tile& t, uint32_t sm, int parts, int part, int warp,
                                          int lane) {
  constexpr int kLanes = BN / 4, kStep = 8 * (32 / kLanes), kRows = 2;   // lanes of a row (four columns each), rows
  const int r1 = t.rows * (part + 1) / parts, col = lane % kLanes * 4;   // of a pass, rows a lane has under way
  for (int r0 = t.rows * part / parts + warp * (32 / kLanes) + lane / kLanes; r0 < r1; r0 += kStep * kRows) {
    float v[kRows][kMaxParts][4];                       // (every load under way at once: one takes some 300 clocks)
#pragma unroll
    for (int u = 0; u < kRows; ++u)
#pragma unroll
      for (int i = 0; i < kMaxParts; ++i)
        if (i < parts && r0 + u * kStep < r1)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[u][i][0]), "=f"(v[u][i][1]), "=f"(v[u][i][2]), "=f"(v[u][i][3])
                       : "r"(map_to(sm + ((r0 + u * kStep) * (BN + 4) + col) * 4, i)));
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * kStep;
      if (r >= r1 || t.n0 + col >= p.N) continue;
      float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kMaxParts; ++i)
        if (i < parts)
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] += v[u][i][j];
      const int64_t at = (int64_t)(t.row0 + r) * p.N + t.n0 + col;
      if (p.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(f32_to_bf16_bits(y[0]) | f32_to_bf16_bits(y[1]) << 16,
                       f32_to_bf16_bits(y[2]) | f32_to_bf16_bits(y[3]) << 16);
    }
  }
}

// SPLIT: the CTAs of a cluster share a tile, each a run of its blocks of inputs, and each sums and stores a part of
// its rows.  The launcher gives every tile a cluster, so a CTA has at most one.
template <int BN, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(Cfg<BN, PAIR>::kThreads, 1) fp8_tc_kernel(const __grid_constant__ Maps maps, const Fp8Matmul p) {
  using C = Cfg<BN, PAIR>;
  static_assert(!(PAIR && SPLIT), "one kind of cluster");
  static_assert(kTileM * (BN + 4) * 4 <= C::kStages * C::kStage || !SPLIT, "a tile's sums take the stages' place");
  constexpr int kCols = BN / (C::kEpiWarps / 4);         // columns of an epilogue thread
  constexpr int kEpiWarps = C::kEpiWarps;
  constexpr int kRows = kTileM * C::kCtas;              // rows of a tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sm = (smem_addr(smem_raw) + 1023) & ~1023u;
  int* pre = reinterpret_cast<int*>(smem_raw + (sm - smem_addr(smem_raw)) + C::kPre);   // [E + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int parts = SPLIT ? (int)cluster_size() : 1, part = SPLIT ? (int)cluster_rank() : 0;
  const int worker = blockIdx.x / (C::kCtas * parts), workers = gridDim.x / (C::kCtas * parts);
  if (threadIdx.x == 0) {
    auto init = [&](int at, int n, uint32_t count) {
      for (int i = 0; i < n; ++i)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sm + at + 8 * i), "r"(count) : "memory");
    };
    init(C::kFull, C::kStages, 1);
    init(C::kEmpty, C::kStages, C::kSplit);
    init(C::kDFull, C::kSplit * C::kBufs, 1);
    init(C::kDEmpty, C::kSplit * C::kBufs, kEpiWarps / C::kSplit * C::kCtas);
    init(C::kSFull, kRing, 32);
    init(C::kSEmpty, kRing, kEpiWarps);
    fence_barrier_init();
  }
  if (warp == 1) {
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem_raw + (sm - smem_addr(smem_raw)) + C::kTmem);
    if (PAIR) {
      tmem_alloc_pair(slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(slot, 512);
      tmem_relinquish();
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");    // launched while the kernel before it may still run
  if (warp == 2) {                                      // row tiles of the experts before each
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      int n = 0;
      if (e0 + lane < p.E) {
        int64_t lo, hi;
        expert_rows(p, e0 + lane, lo, hi);
        n = (int)((hi - lo + kRows - 1) / kRows);
      }
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
      }
      if (e0 + lane < p.E) pre[e0 + lane] = before + inc - n;
      before += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    if (lane == 0) pre[p.E] = before;
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();                             // both CTAs' barriers are initialised
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(sm + C::kTmem));
  const int ntiles = (p.N + BN - 1) / BN;
  const int total = SPLIT ? min(pre[p.E] * ntiles, workers) : pre[p.E] * ntiles;
  const int kall = (p.K + 127) / 128, nblocks = (p.N + 127) / 128;
  const int kb0 = SPLIT ? part * part_blocks(kall, parts) : 0;   // this CTA's blocks: kblocks from kb0 on
  const int kblocks = SPLIT ? min(part_blocks(kall, parts), kall - kb0) : kall;

  if (warp < kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    if (BN == 256) regs_inc<kRegsEpi>();
    // Columns (warp / 4) kCols .. of the accumulator.  A pair's half h holds 64 weight rows of each CTA's 128: the
    // second 64 columns then are 128 further in the tile, and belong to the second weight tile.
    const int g = warp >> 2, h = C::kSplit == 2 ? g : 0;
    const int col = PAIR ? h * 64 : g * kCols;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + g * kCols;
    const uint32_t d_full = sm + C::kDFull + 8 * h * C::kBufs;
    const uint32_t d_empty = (PAIR ? map_to(sm + C::kDEmpty, 0) : sm + C::kDEmpty) + 8 * h * C::kBufs;
    const uint32_t my_a = sm + C::kScales + ((warp & 3) * 32 + lane) * 16;
    const uint32_t my_b = sm + C::kScales + kTileM * 16;
    uint32_t slot = 0, s_phase = 0, buf = 0, phase = 0;
    bool whole_tile = false;
    for (int tt = worker; tt < total; tt += workers) {
      float acc[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
      if (!warp_wait(sm + C::kSFull + 8 * slot, s_phase)) goto leave;
      float sa = lds_f32(my_a + slot * C::kScaleSlot), sb = lds_f32(my_b + slot * C::kScaleSlot);
      float sb2 = PAIR ? lds_f32(my_b + slot * C::kScaleSlot + 16) : 0.0f;
      bool seen = bar_peek(d_full + 8 * buf, phase);    // the block's accumulator was found complete
#pragma unroll 1
      for (int kb = 0;;) {
        const float sc = sa * sb, sc2 = PAIR ? sa * sb2 : 0.0f;
        const uint32_t at = lane_base + buf * BN, done = d_empty + 8 * buf;
        if (!__all_sync(0xFFFFFFFFu, seen) && !warp_wait(d_full + 8 * buf, phase)) goto leave;
        tc_fence_after();
        if (++buf == C::kBufs) {
          buf = 0;
          phase ^= 1;
        }
        ++kb;
        // Sixteen columns load while the sixteen before them are added; under the last ones' additions the next
        // block's scales and accumulator are looked for.
        float d[2][16];
        tmem_ld16(at, d[0]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          if (c + 16 < kCols) {
            tmem_ld16(at + c + 16, d[(c / 16 + 1) & 1]);
          } else {
            tc_fence_before();                          // the accumulator is free again
            if (lane == 0) {
              if (PAIR)
                arrive_remote(done);
              else
                bar_arrive(done);
            }
            const uint32_t next = slot * C::kScaleSlot + (kb & 3) * 4;   // (at a group's end read again below)
            sa = lds_f32(my_a + next);
            sb = lds_f32(my_b + next);
            if (PAIR) sb2 = lds_f32(my_b + next + 16);
            seen = bar_peek(d_full + 8 * buf, phase);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) fma_acc(acc[c + j], d[(c / 16) & 1][j], PAIR && c >= 64 ? sc2 : sc);
          if (c + 16 < kCols) tmem_wait_ld();
        }
        const bool last = kb == kblocks;
        if ((kb & 3) == 0 || last) {                    // done with this slot's scales
          __syncwarp();
          if (lane == 0) bar_arrive(sm + C::kSEmpty + 8 * slot);
          if (++slot == kRing) {
            slot = 0;
            s_phase ^= 1;
          }
          if (last) break;
          if (!warp_wait(sm + C::kSFull + 8 * slot, s_phase)) goto leave;
          sa = lds_f32(my_a + slot * C::kScaleSlot);
          sb = lds_f32(my_b + slot * C::kScaleSlot);
          if (PAIR) sb2 = lds_f32(my_b + slot * C::kScaleSlot + 16);
        }
      }
      if (SPLIT) {                                      // where the stages were: all loads and MMAs are done
        const uint32_t row = sm + ((warp & 3) * 32 + lane) * (BN + 4) * 4 + col * 4;
#pragma unroll
        for (int c = 0; c < kCols; c += 4)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(row + 4 * c), "f"(acc[c]), "f"(acc[c + 1]),
                       "f"(acc[c + 2]), "f"(acc[c + 3])
                       : "memory");
        whole_tile = true;
      } else {
        const Tile t = find_tile(p, pre, ntiles, BN, kRows, tt);
        const int r0 = kTileM * rank + (warp & 3) * 32;
        const int esize = p.out_f32 ? 4 : 2;
        uint8_t* row0 = static_cast<uint8_t*>(p.out) + ((int64_t)(t.row0 + r0) * p.N + t.n0) * esize;
        const auto column = [&](int c) { return col + c + (PAIR && c >= 64 ? 64 : 0); };
        const uint32_t stage = sm + C::kOut + warp * 2048;
        if (p.out_f32)
          store_rows<kCols, true>(acc, stage, row0, (int64_t)p.N * 4, t.rows - r0, p.N - t.n0, lane, column);
        else
          store_rows<kCols, false>(acc, stage, row0, (int64_t)p.N * 2, t.rows - r0, p.N - t.n0, lane, column);
      }
    }
  leave:
    if (SPLIT) {
      cluster_sync();                                   // the parts' sums are in place
      if (whole_tile) sum_parts<BN>(p, find_tile(p, pre, ntiles, BN, kRows, worker), sm, parts, part, warp, lane);
    }
    all_done<PAIR || SPLIT, C::kThreads>();
    if (warp == 1) {
      if (PAIR)
        tmem_dealloc_pair(tmem, 512);
      else
        tmem_dealloc(tmem, 512);
    }
    return;
  }
  if (BN == 256) regs_dec<kRegsRest>();
  if (warp < kEpiWarps + C::kTmaWarps) {
    // ------------------------------------------------------------ TMA
    const uint32_t full0 = PAIR ? map_to(sm + C::kFull, 0) : sm + C::kFull;
    const bool leader = elect_one();
    const int first = warp - kEpiWarps;
    int q = first, s = first, kb = first;
    uint32_t phase = 1;
    bool ok = true;
    for (int tt = worker; tt < total && ok; tt += workers) {
      const Tile t = find_tile(p, pre, ntiles, BN, kRows, tt);
      const int box = box_of(t.rows - rank * kTileM), other = PAIR ? box_of(t.rows - (1 - rank) * kTileM) : 0;
      const CUtensorMap* amap = &maps.a[box >> 6];                      // 32, 64, 128
      const int arow = t.row0 + rank * kTileM, brow = t.e * p.N + t.n0 + rank * C::kBRows;
      const uint32_t bytes = (box + other) * 128 + C::kCtas * C::kBBytes;
      for (; kb < kblocks; kb += C::kTmaWarps, q += C::kTmaWarps) {
        if (!warp_wait(sm + C::kEmpty + 8 * s, phase)) {
          ok = false;
          break;
        }
        if (leader) {
          const uint32_t st = sm + s * C::kStage, bar = full0 + 8 * s;
          if (rank == 0) bar_expect(sm + C::kFull + 8 * s, bytes);
          tma_load_to<PAIR>(st + kABytes, &maps.b, (kb0 + kb) * 128, brow, bar);
          if (!PAIR || box > 0) tma_load_to<PAIR>(st, amap, (kb0 + kb) * 128, arow, bar);
        }
        __syncwarp();
        if ((s += C::kTmaWarps) >= C::kStages) {
          s -= C::kStages;
          phase ^= 1;
        }
      }
      kb -= kblocks;
    }
    // Leave no copy in flight: CTA 0 waits for its stages' bytes (both halves of a pair's); CTA 1's
    // copies complete on those same barriers, so it waits for the MMA commits of its last stages.
    for (int j = max(first, q - C::kStages); j < q; j += C::kTmaWarps)
      bar_wait(sm + (rank == 0 ? C::kFull : C::kEmpty) + 8 * (j % C::kStages), (j / C::kStages) & 1);
    __syncwarp();
  } else if (warp < kEpiWarps + C::kTmaWarps + kMmaWarps) {
    // ------------------------------------------------------------ MMA
    // Warp m takes half m of every block (BN = 256) or the whole of every other block: they do not depend on
    // one another, and the waits and the issue of one take a warp about 460 clocks.
    constexpr int kN = BN / C::kSplit, kStep = kMmaWarps / C::kSplit;
    constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
    const int m = warp - (kEpiWarps + C::kTmaWarps), h = C::kSplit == 2 ? m : 0, first = C::kSplit == 2 ? 0 : m;
    const bool leader = elect_one();
    const uint64_t desc0 = smem_desc_sw128(sm);
    const uint32_t boff = (kABytes + h * (C::kBBytes / C::kSplit)) >> 4;
    const uint32_t d_full = sm + C::kDFull + 8 * h * C::kBufs, d_empty = sm + C::kDEmpty + 8 * h * C::kBufs;
    const int steps = rank == 0 && worker < total ? ((total - worker + workers - 1) / workers) * kblocks : 0;
    uint32_t s = first, phase = 0, buf = first, d_phase = 1;
    int q = first;
#pragma unroll 1
    for (; q < steps; q += kStep) {
      if (!warp_wait(d_empty + 8 * buf, d_phase) || !warp_wait(sm + C::kFull + 8 * s, phase)) break;
      tc_fence_after();
      if (leader) {
        const uint64_t da = desc0 + s * (C::kStage >> 4), db = da + boff;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_f8<PAIR>(tmem + buf * BN + h * kN, da + 2 * k, db + 2 * k, idesc, k != 0);
        commit<PAIR>(d_full + 8 * buf);
        commit<PAIR>(sm + C::kEmpty + 8 * s);
      }
      __syncwarp();
      if ((s += kStep) >= C::kStages) {
        s -= C::kStages;
        phase ^= 1;
      }
      if ((buf += kStep) >= C::kBufs) {
        buf -= C::kBufs;
        d_phase ^= 1;
      }
    }
    const int last = q - kStep;                         // the last block issued
    // Do not free tensor memory while MMAs may still run (matters only on an error path).
    if (last >= 0) bar_wait(sm + C::kEmpty + 8 * (last % C::kStages), (last / C::kStages) & 1);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scales
    // The a_scales of this CTA's 128 rows (4 a lane) and the b_scales of the tile's one or two weight tiles, four
    // blocks at a time, copied to shared memory ahead of the epilogue, which has no registers for loads under way.
    const bool whole = (kall & 3) == 0 && (reinterpret_cast<uintptr_t>(p.a_scales) & 15) == 0;
    int slot = 0;
    uint32_t phase = 1;
    bool ok = true;
    for (int tt = worker; tt < total && ok; tt += workers) {
      const Tile t = find_tile(p, pre, ntiles, BN, kRows, tt);
      const int mine = t.rows - kTileM * rank - lane;   // rows of the tile from this lane's first on
      const float* as = p.a_scales + (int64_t)(t.row0 + kTileM * rank + lane) * kall + kb0;
      const float* bs =
          p.b_scales + ((int64_t)t.e * nblocks + min(t.n0 / 128 + (lane >> 2), nblocks - 1)) * kall + kb0 + (lane & 3);
      for (int kb = 0; kb < kblocks; kb += 4) {
        if (!warp_wait(sm + C::kSEmpty + 8 * slot, phase)) {
          ok = false;
          break;
        }
        const uint32_t dst = sm + C::kScales + slot * C::kScaleSlot;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (32 * j < mine) {
            const float* src = as + (int64_t)(32 * j) * kall + kb;
            if (whole) {
              cp_async16(dst + (32 * j + lane) * 16, src);
            } else {
              for (int i = 0; i < min(4, kblocks - kb); ++i) cp_async4(dst + (32 * j + lane) * 16 + 4 * i, src + i);
            }
          }
        if (lane < 4 * C::kScaleHalves && kb + (lane & 3) < kblocks)
          cp_async4(dst + kTileM * 16 + 4 * lane, bs + kb);
        cp_async_arrive(sm + C::kSFull + 8 * slot);
        if (++slot == kRing) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
  if (SPLIT) cluster_sync();
  all_done<PAIR || SPLIT, C::kThreads>();
}

// Row tiles at most: the offsets are not known here.
int64_t most_row_tiles(const Fp8Matmul& p, int rows) {
  return p.offsets ? (p.M + (rows - 1) * std::min<int64_t>(p.E, p.M)) / rows : (p.M + rows - 1) / rows;
}

// Clusters that run at once, 0 where the query fails (which then is no error of the call's).
int active_clusters(const void* kern, const cudaLaunchConfig_t& cfg) {
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess) return n;
  cudaGetLastError();
  return 0;
}

// parts: CTAs that share a tile's inputs (SPLIT; else 1).
template <int BN, bool PAIR, bool SPLIT>
int launch_tc(const Fp8Matmul& p, int dev, int num_sms, int parts, cudaStream_t s) {
  using C = Cfg<BN, PAIR>;
  Maps maps;
  const uint64_t da[2] = {(uint64_t)p.K, (uint64_t)p.M}, db[2] = {(uint64_t)p.K, (uint64_t)p.E * p.N};
  const uint64_t st[1] = {(uint64_t)p.K};
  const uint32_t bb[2] = {128, C::kBRows};
  int rc = 0;
  for (int i = 0; i < 3 && !rc; ++i) {
    const uint32_t ba[2] = {128, 32u << i};
    rc = make_tensor_map(&maps.a[i], 2, p.a, da, st, ba, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (!rc) rc = make_tensor_map(&maps.b, 2, p.b, db, st, bb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc) return rc;
  auto kern = fp8_tc_kernel<BN, PAIR, SPLIT>;
  if (BN == 256) {                                      // what the register split draws on
    static PerDevice known;
    const int regs = known.get(dev, [&] {
      cudaFuncAttributes a{};
      return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
    });
    if ((regs + 7) / 8 * 8 < kRegsLaunch) return -(int)cudaErrorLaunchOutOfResources;
  }
  cudaError_t err = set_smem_limit(reinterpret_cast<const void*>(kern), C::kSmem);
  if (err != cudaSuccess) return -(int)err;
  const int64_t most = most_row_tiles(p, kTileM * C::kCtas) * ((p.N + BN - 1) / BN);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::kCtas * parts;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)num_sms / C::kCtas * C::kCtas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR || SPLIT ? 2 : 1;
  int workers = num_sms;
  if (PAIR) {                                           // pairs resident at once
    static PerDevice known;
    const int pairs = known.get(dev, [&] { return active_clusters(reinterpret_cast<const void*>(kern), cfg); });
    if (pairs < 1) return -(int)cudaErrorLaunchOutOfResources;
    workers = pairs;
  }
  cfg.gridDim = dim3((unsigned)(SPLIT ? most * parts : C::kCtas * std::min<int64_t>(most, workers)));
  err = cudaLaunchKernelEx(&cfg, kern, maps, p);
  if (err == cudaSuccess) err = cudaGetLastError();
  return err == cudaSuccess ? 1 : -(int)err;
}

// Clusters of `parts` CTAs that run at once (fewer than SMs / parts: a cluster stays within one of the GPU's groups
// of SMs; of eight, 64 rows x 1024 x 8192 took a second wave).
int resident_clusters(int dev, int parts) {
  static PerDevice known[kMaxParts + 1];
  return known[parts].get(dev, [&] {
    using C = Cfg<64, false>;
    const void* kern = reinterpret_cast<const void*>(fp8_tc_kernel<64, false, true>);
    if (set_smem_limit(kern, C::kSmem) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)parts);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return active_clusters(kern, cfg);
  });
}

}  // namespace

// Reads and clears this file's device status.
cudaError_t fp8_take_status(int* v) {
  const int zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(v, g_status, sizeof(int));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
}

// The tile: the one with the least estimated time, fixed + waves * blocks of 128 inputs * the time of a block, from
// measurements (us): a lone wave's blocks are bound by one CTA's chain of steps, more waves' by the L2's rate.  Tiles
// shared by a cluster of CTAs, for calls of a few tiles and long rows, pay for joining the sums.  Both sides
// measured, K = 5120 (us; 64 / 128 / pair): 64 rows, N = 5120: 10.9 / 13.1 / 20.5; 256 rows: 20.6 / 13.8 / 21.6;
// 4096 rows: 156 / 111 / 100; 2048 rows over 32 experts: 206 / 145 / 197; 8192 over 32: 396 / 298 / 297 (256 rows an
// expert, many of which take two of the pair's tiles; the estimate, 225 and 220, leaves that out on both sides); 65536
// over 256: 3785 / 2473 / 2937; 65787 over 32: 2779 / 1792 / 1597; 64
// rows, N = 2560: 10.5, two or three CTAs a tile 9.0 / 8.6; N = 512: 10.5, five 6.8; N = 1024, K = 8192: 14.7, two
// / four / eight 11.1 / 8.4 / 8.1.  The row tiles of several experts are not known here: an expert's last is taken
// to be half full.
int launch_fp8_matmul(const Fp8Matmul& p, const Fp8Tile& forced, int dev, int num_sms, cudaStream_t s) {
  struct Form {
    int tile_m, bn;
    double fixed, lone, loaded, join;
  };
  static constexpr Form kForms[3] = {{kTileM, 64, 4.2, 0.166, 0.225, 1.5},
                                     {kTileM, 128, 4.9, 0.215, 0.25, 2.0},
                                     {2 * kTileM, 256, 7.0, 0.37, 0.41, 0.0}};
  const int kall = (p.K + 127) / 128;
  const int64_t spread = p.offsets ? p.E / 2 : 0;
  // Every part has blocks, and the tiles run at once.
  const auto parts_ok = [&](int bn, int parts, int64_t clusters) {
    return (parts - 1) * part_blocks(kall, parts) < kall && most_row_tiles(p, kTileM) * ((p.N + bn - 1) / bn) <= clusters;
  };
  int bn = 0, parts = 1;
  double best = 0.0;
  for (const Form& f : kForms) {
    const int64_t mt = std::min<int64_t>(p.M, (p.M + f.tile_m - 1) / f.tile_m + spread);
    const int workers = f.bn == 256 ? num_sms / 2 : num_sms;
    const int64_t waves = (mt * ((p.N + f.bn - 1) / f.bn) + workers - 1) / workers;
    const double c = f.fixed + (waves == 1 ? f.lone : f.loaded * (double)waves) * kall;
    if (bn == 0 || c < best) {
      best = c;
      bn = f.bn;
      parts = 1;
    }
    for (int n = 2; n <= kMaxParts && f.bn < 256; ++n) {
      const double cn = f.fixed + f.join + f.lone * part_blocks(kall, n);
      if (cn < best && parts_ok(f.bn, n, resident_clusters(dev, n))) {
        best = cn;
        bn = f.bn;
        parts = n;
      }
    }
  }
  if (forced.bn) {
    bn = forced.bn;
    parts = forced.parts;
    while (parts > 1 && !parts_ok(bn, parts, 1 << 14)) --parts;
  } else if (fp8_few_wanted(p, num_sms)) {
    return launch_fp8_few(p, s);
  }
  if (bn == 256) return launch_tc<256, true, false>(p, dev, num_sms, 1, s);
  if (bn == 128)
    return parts > 1 ? launch_tc<128, false, true>(p, dev, num_sms, parts, s) : launch_tc<128, false, false>(p, dev, num_sms, 1, s);
  return parts > 1 ? launch_tc<64, false, true>(p, dev, num_sms, parts, s) : launch_tc<64, false, false>(p, dev, num_sms, 1, s);
}

}  // namespace moe
