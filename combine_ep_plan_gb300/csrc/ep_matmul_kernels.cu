// ep_matmul_kernels.cu — products of 8-bit codes with the experts' 8-bit
// weights, with a scale for each row and each channel:
//
//   out[r,n] = round( a_scale[s] * w_scale[e,n] * sum_k a[s,k] * w[e,n,k] ),  s = rows[r] (or r)
//
// for the rows r of expert e, offsets[e] <= r < offsets[e+1]: the expanded
// layout of the plan.  A row with s = -1 is zero.
//
// Arithmetic.  This GPU's tensor cores have little rate for 8-bit integers
// (157 TOP/s measured); fp16 holds every 8-bit code exactly, so where there are
// rows enough the codes are widened to fp16 on the way into the tensor cores
// (tcgen05.mma kind::f16), which sum in fp32.  Every product is at most 2^14, so a
// running sum is an exact integer as long as it stays within 2^24: for K <= 1024
// whatever the codes, for longer sums unless nearly all codes are at the end of
// their range with one sign; beyond it each step rounds like any fp32 sum.
//
// Three kernels, by the mean number of rows per expert (measured at 64 experts,
// 7168 -> 4096, each rule beside its constant):
//   a handful   integer products straight from registers; the weights' stream
//               is all (64 tokens top-6: 332 us, 5.7 TB/s of weights; in a row 308);
//   up to 120   rows in tensor memory, weights widened in shared memory, 256
//               channels x 128 rows a tile (1024 tokens: 400 us);
//   more        CTA pairs, 256 channels x 256 rows (16384 tokens: 3.53 ms, 1636
//               TFLOP/s; in a row 3.6 ms, under the power limit).
// Times here are of one launch with cold caches, unless they are called in a row.
//
// The pairs' kernel.  The weights are the A operand (128 channels = 128 lanes of
// tensor memory per CTA), the rows the B operand (N columns).  Widened weights go
// from registers into tensor memory, not back through shared memory: per 16
// steps of k an SM then moves 16 KB through its shared memory, against 12 KB more
// otherwise, in the 128 clocks its products take.  A tile's time does not depend
// on its rows (a product with its A operand in tensor memory takes no less than
// about 128 clocks), so the tail of a group costs a whole tile.
//
// Roles of a CTA's 28 warps: warp 0 loads weight codes (TMA, 128 channels x 128
// k per stage); warp 1 issues the products; warps 4-11 widen weights into tensor
// memory; warps 12-19 load the rows' codes (16-byte loads, any row order), widen
// them into shared memory (K-major, 128-byte swizzle); warps 20-27 scale,
// round and store finished tiles.  What bounds it: the instructions of the
// widening, five for four codes, share the issue slots with the one thread that
// keeps the tensor cores fed.  CTAs are persistent and take tiles in turn; the
// row tiles of one expert lie next to one another in that order, so that its
// weights are read from L2.
#include <atomic>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ep_internal.cuh"
#include "ep_plan.h"

namespace ep {
namespace {

constexpr int kStageK = 128;                // k per stage
constexpr int kChannels = 128;              // channels per CTA
constexpr int kWBytes = kChannels * kStageK;  // a stage of weight codes
constexpr int kStages = 4;                  // widened stages
constexpr int kACols = 64;                  // tensor-memory columns of a widened weight stage
constexpr int kABase = 512 - kStages * kACols;

// ---- PTX ----

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// What the CTAs of a pair hand to the leader: an arrival on its barrier, at cluster
// scope, behind a release of the widened rows in shared memory (weights and results
// in tensor memory are ordered by tcgen05's own fences); the leader waits at cluster
// scope and acquires.  A release of all memory would wait for the loads of the next
// rows too: 2045 tokens top-6 387 us against 301; arrivals and waits that name no
// scope, and so order nothing between two CTAs by the letter, 298.
__device__ __forceinline__ void mbar_arrive_leader(uint32_t bar) {
  asm volatile(
      "{\n .reg .b32 ra;\n mapa.shared::cluster.u32 ra, %0, 0;\n"
      " mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [ra];\n}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void release_shared() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
__device__ __forceinline__ void acquire_shared() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// What a CTA's copies and products in flight are waited for before it ends,
// whatever the limit of its other waits.
constexpr unsigned long long kDrainNs = 2000000000ull;

// Every wait ends: after limit_ns it records a timeout, marks the CTA dead
// (its other waits then give up too) and returns false.
struct Waiter {
  unsigned* status;
  volatile int* dead;
  unsigned long long limit_ns;
  __device__ bool slow(uint32_t bar, uint32_t parity, bool heed_dead, unsigned long long limit) const {
    unsigned long long t0 = 0;
    for (;;) {
      for (int i = 0; i < 64; ++i)  // the clock is slow to read
        if (mbar_try(bar, parity)) return true;
      if (heed_dead && *dead) return false;
      if (t0 == 0) t0 = now_ns();
      if (now_ns() - t0 > limit) {
        atomicOr(status, kStTimeout);
        *dead = 1;
        return false;
      }
    }
  }
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    return mbar_try(bar, parity) || slow(bar, parity, true, limit_ns);
  }
  // For what is in flight, also in a dead CTA.
  __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) const {
    if (!mbar_try(bar, parity)) slow(bar, parity, false, kDrainNs);
  }
  // For an arrival from the other CTA.
  __device__ __forceinline__ bool cluster(uint32_t bar, uint32_t parity) const {
    return mbar_try_cluster(bar, parity) || (slow(bar, parity, true, limit_ns) && mbar_try_cluster(bar, parity));
  }
  // By a whole warp, with one answer for it.
  __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
    return __all_sync(~0u, (*this)(bar, parity));
  }
};

__device__ __forceinline__ void tma_weights(uint32_t dst, const CUtensorMap* map, int k, int n, int e, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(k), "r"(n), "r"(e)
      : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t slot) {
  if (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base) {
  if (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(base));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (+)= A (tensor memory) * B (shared memory)
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// Arrives on the barrier (of both CTAs of a pair) when every product issued so far is done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// ... of a pair's products, on the barrier of this CTA alone.
__device__ __forceinline__ void mma_commit_here(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 256 bits, four times: lane 4g + t of the warp gives registers 4b and
// 4b + 1 to tensor-memory lane g, columns 8b + 2t and 8b + 2t + 1, and registers 4b + 2
// and 4b + 3 to lane g + 8.
__device__ __forceinline__ void tmem_st16x256(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 columns of them.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Two sums times their row's scales, then the channel's, two products an instruction.
__device__ __forceinline__ void scale2(uint32_t s0, uint32_t s1, float a0, float a1, float w, float& y0, float& y1) {
  asm("{\n .reg .b64 s, a, w;\n mov.b64 s, {%2, %3};\n mov.b64 a, {%4, %5};\n mov.b64 w, {%6, %6};\n"
      " mul.rn.f32x2 s, s, a;\n mul.rn.f32x2 s, s, w;\n mov.b64 {%0, %1}, s;\n}"
      : "=f"(y0), "=f"(y1)
      : "r"(s0), "r"(s1), "f"(a0), "f"(a1), "f"(w));
}

// Four codes to four halves: the byte u = code + 128 under the exponent of
// 1024 is the half 1024 + u; less 1152 it is the code, exactly.
__device__ __forceinline__ void widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = codes ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const uint32_t bias = 0x64806480u;
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&bias));
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&bias));
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Through L1: eight lanes share a 128-byte line.  (Loads that do not allocate
// there took a third longer in all.)
__device__ __forceinline__ uint4 ld_codes(const int8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Rows of codes are brought to L2 this many bytes before they are loaded: the
// channel tiles of the same rows run side by side, and without it all of them
// wait for memory at every piece (64 experts, 7168 -> 4096: 24 rows each 462 us,
// 374 with it; 96 rows 493 and 412; 384 rows 1394 and 1277; 1024 bytes do the same,
// 2048 are too far for the first).
constexpr int kAhead = 512;
__device__ __forceinline__ void prefetch_line(const int8_t* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ int clamp_row(int v, int64_t rows) {
  return v < 0 ? 0 : v > rows ? static_cast<int>(rows) : v;
}

// A B operand in shared memory: rows of 64 halves (128 bytes), swizzled by 128
// bytes, k contiguous; `low` is b_desc_low() of its address, plus bytes / 16.
__device__ __forceinline__ uint32_t b_desc_low(uint32_t addr) { return ((addr >> 4) & 0x3fff) | (1u << 16); }
__device__ __forceinline__ uint64_t b_desc(uint32_t low) {
  return static_cast<uint64_t>(low) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The warp's number, as a value the compiler knows to be the same in its lanes
// (it then keeps addresses in uniform registers, and spills none).
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(~0u, static_cast<int>(threadIdx.x >> 5), 0); }

// ---- tiles ----

struct Tile {
  int e, n0;     // expert, first channel (of the CTA pair)
  int r0, rows;  // first output row, rows
};

// The experts' rows in shared memory: [E+1] row tiles before each expert, then
// [E+1] first rows.
struct Groups {
  int* tiles;
  int* rows;
  __device__ Groups(void* at, int E) : tiles(static_cast<int*>(at)), rows(tiles + E + 1) {}
  static size_t bytes(int E) { return 2 * sizeof(int) * (E + 1); }
};

// Row tiles of nt rows that ascending offsets make at most: every group but one
// may add a tile to those of the rows in a row, and every tile has a row.
__host__ __device__ __forceinline__ int64_t most_row_tiles(int64_t rows, int E, int nt) {
  const int64_t most = (rows + nt - 1) / nt + E - 1;
  return most < rows ? most : rows;
}

// By one warp.  Offsets that do not ascend are held to as many tiles as ascending
// ones make: tile indices stay within 32 bits, and a grid that has a cluster for
// each tile has one for each of theirs.
__device__ __forceinline__ void find_groups(const MatmulDev& d, const Groups& g, int NT, int lane) {
  const int most = static_cast<int>(most_row_tiles(d.out_rows, d.E, NT));
  int sum = 0;
  for (int e0 = 0; e0 < d.E; e0 += 32) {
    const int e = e0 + lane;
    int tiles = 0;
    if (e < d.E) {
      const int r0 = d.offsets ? clamp_row(d.offsets[e], d.out_rows) : 0;
      const int r1 = d.offsets ? clamp_row(d.offsets[e + 1], d.out_rows) : static_cast<int>(d.out_rows);
      tiles = r1 > r0 ? (r1 - r0 + NT - 1) / NT : 0;
      g.rows[e] = r0;
      if (e == d.E - 1) g.rows[d.E] = r1;
    }
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += v;
    }
    if (e < d.E) g.tiles[e + 1] = min(sum + upto, most);
    sum = min(sum + __shfl_sync(~0u, upto, 31), most);
  }
  if (lane == 0) g.tiles[0] = 0;
  if (blockIdx.x == 0 && lane == 0 && d.offsets && d.offsets[d.E] > d.out_rows) atomicOr(d.status, kStCapacity);
}

// Walks the tiles start, start + step, ... of all, tiles of NT rows x CH
// channels; a tile's index counts expert, channel tile and row tile, row tiles
// fastest.
template <int NT, int CH>
struct Cursor {
  const MatmulDev& d;
  const Groups& g;
  unsigned t, stride;
  int e = 0;
  __device__ Cursor(const MatmulDev& dev, const Groups& groups, unsigned start, unsigned step)
      : d(dev), g(groups), t(start), stride(step) {}
  __device__ unsigned channel_tiles() const { return (d.N + CH - 1) / CH; }
  __device__ unsigned all() const { return g.tiles[d.E] * channel_tiles(); }
  __device__ __forceinline__ bool next(Tile& out) {
    if (t >= all()) return false;
    const unsigned nch = channel_tiles();
    while (t >= g.tiles[e + 1] * nch) ++e;
    const unsigned before = g.tiles[e], row_tiles = g.tiles[e + 1] - before;
    const unsigned l = t - before * nch;
    const unsigned c = row_tiles == 1 ? l : l / row_tiles;
    out.e = e;
    out.n0 = c * CH;
    out.r0 = g.rows[e] + (l - c * row_tiles) * NT;
    out.rows = min(NT, g.rows[e + 1] - out.r0);
    t += stride;
    return true;
  }
};

__device__ __forceinline__ int source_row(const MatmulDev& d, int r) {
  const int s = d.rows ? d.rows[r] : r;
  return s < d.a_rows ? s : -1;
}

// ---- CTA pairs: 256 channels x 256 rows ----

constexpr int kPairThreads = 896;
constexpr int kRowsPair = 256;              // rows of a tile
constexpr int kRowsCta = kRowsPair / 2;     // ... widened by one CTA
constexpr int kW = 4;                       // stages of weight codes
constexpr int kHalf = kRowsCta * 128;       // the first 64 k of a stage of widened rows
constexpr int kBBytes = 2 * kHalf;

struct PairShape {
  static constexpr int kCodes = 0, kB = kW * kWBytes;
  static constexpr int kScale = kB + kStages * kBBytes;   // [8][128] row scales, for each storing warp its own
  static constexpr int kZero = kScale + 8 * kRowsCta * 4;  // [8][4] zero rows
  static constexpr int kBars = kZero + 8 * (kRowsCta / 32) * 4;
  static constexpr int kNumBars = 2 * kW + 2 * kStages + 3;
  static constexpr int kMisc = kBars + kNumBars * 8;      // tensor-memory base, dead flag
  static constexpr int kGroups = kMisc + 16;
  static size_t bytes(int E) { return 1024 + kGroups + Groups::bytes(E); }
};

template <typename Out>
__global__ void __launch_bounds__(kPairThreads, 1) ep_matmul_pair_kernel(const __grid_constant__ CUtensorMap wmap, MatmulDev d) {
  using L = PairShape;
  extern __shared__ uint8_t raw[];
  const uint32_t raw_at = smem_u32(raw);
  uint8_t* smem = raw + ((1024 - (raw_at & 1023)) & 1023);
  const uint32_t at = smem_u32(smem);
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

  // barriers
  const uint32_t bars = at + L::kBars;
  auto w_full = [&](int s) { return bars + 8 * s; };                     // weight codes landed
  auto w_empty = [&](int s) { return bars + 8 * (kW + s); };             // ... and were read
  auto full = [&](int s) { return bars + 8 * (2 * kW + s); };            // widened stage ready (the leader's)
  auto empty = [&](int s) { return bars + 8 * (2 * kW + kStages + s); }; // ... and used
  const uint32_t d_full = bars + 8 * (2 * kW + 2 * kStages);             // the tile's products are done
  const uint32_t d_empty = d_full + 8;                                   // ... and were taken (the leader's)
  const uint32_t drained = d_full + 16;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  const Groups groups(smem + L::kGroups, d.E);
  const Waiter wait{d.status, reinterpret_cast<volatile int*>(misc + 1), d.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kW; ++s) {
      mbar_init(w_full(s), 1);
      mbar_init(w_empty(s), 4);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 2 * 8);
      mbar_init(empty(s), 1);
    }
    mbar_init(d_full, 1);
    mbar_init(d_empty, 2 * 8);
    mbar_init(drained, 1);
    misc[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<2>(at + L::kMisc);
  pdl_wait();
  if (warp == 2) find_groups(d, groups, kRowsPair, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int k_stages = (d.K + kStageK - 1) / kStageK;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  Tile tile;
  Cursor<kRowsPair, 2 * kChannels> cur(d, groups, blockIdx.x / 2, gridDim.x / 2);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 && lane == 0) {
      // weight codes
      uint32_t it = 0;
      bool ok = true;
      while (ok && cur.next(tile)) {
        if (d.suppress && blockIdx.x == 0) break;
        for (int k = 0; k < k_stages; ++k, ++it) {
          const int s = it % kW;
          if (!(ok = wait(w_empty(s), (it / kW + 1) & 1))) break;
          mbar_expect(w_full(s), kWBytes);
          tma_weights(at + L::kCodes + s * kWBytes, &wmap, k * kStageK, tile.n0 + static_cast<int>(rank) * kChannels,
                      tile.e, w_full(s));
        }
      }
      // Loads in flight end before the CTA does: those who read them may have given up.
      for (uint32_t i = it > kW ? it - kW : 0; i < it; ++i) wait.drain(w_full(i % kW), (i / kW) & 1);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // products
      uint32_t it = 0, nt = 0;
      bool ok = true;
      while (ok && cur.next(tile)) {
        const int n = (tile.rows + 31) / 32 * 32;
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(2 * kChannels >> 4) << 24);
        if (!(ok = wait.cluster(d_empty, (nt + 1) & 1))) break;
        // What the next stage needs is made ready before this one's last product
        // is issued: between two stages nothing but the commit keeps the tensor
        // cores waiting (4.09 -> 3.75 ms for the prefill's product).
        auto b_at = [&](uint32_t i) { return b_desc_low(at + L::kB + i % kStages * kBBytes); };
        auto a_at = [&](uint32_t i) { return tmem + kABase + i % kStages * kACols; };
        uint32_t a = a_at(it), b = b_at(it), add = 0;
        if (!(ok = wait.cluster(full(it % kStages), (it / kStages) & 1))) break;
        tc_fence_after();
        acquire_shared();
        for (int k = 1; k < k_stages; ++k) {
          bool ready = false;
          uint32_t next_a = 0, next_b = 0;
          const uint32_t done = empty(it % kStages);
          ++it;
#pragma unroll
          for (int i = 0; i < kStageK / 16; ++i) {
            if (i == kStageK / 16 - 2) {
              next_a = a_at(it);
              next_b = b_at(it);
              ready = mbar_try_cluster(full(it % kStages), (it / kStages) & 1);
            }
            mma_f16<2>(tmem, a + i * 8, b_desc(b + (i >> 2) * (kHalf / 16) + (i & 3) * 2), idesc, i == 0 ? add : 1);
          }
          mma_commit<2>(done);
          a = next_a;
          b = next_b;
          add = 1;
          if (!ready && !(ok = wait.cluster(full(it % kStages), (it / kStages) & 1))) break;
          tc_fence_after();
          acquire_shared();
        }
        if (!ok) break;
        const int steps = (d.K - (k_stages - 1) * kStageK) / 16;
        for (int i = 0; i < steps; ++i)
          mma_f16<2>(tmem, a + i * 8, b_desc(b + (i >> 2) * (kHalf / 16) + (i & 3) * 2), idesc, add | i);
        mma_commit<2>(empty(it % kStages));
        ++it;
        mma_commit<2>(d_full);
        ++nt;
      }
      // Products in flight end before tensor memory is given back: those who take them may have given up.
      mma_commit_here(drained);
      wait.drain(drained, 0);
    }
  } else if (warp < 12) {
    // Weights to fp16 in tensor memory: a thread widens one channel, warps 4-7
    // the even stages and 8-11 the odd ones.  The next codes are read, if they
    // are there, while these are on their way to tensor memory.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int row = threadIdx.x & 127;
    uint32_t it = (warp - 4) >> 2;  // of all stages of this CTA's tiles
    // Whether stage `it` exists: tiles are counted as they are reached.
    uint32_t known = 0;
    auto exists = [&](uint32_t i) {
      while (i >= known) {
        if (!cur.next(tile)) return false;
        known += k_stages;
      }
      return true;
    };
    uint4 c[8];
    auto read = [&](int ws) {
      const uint8_t* src = smem + L::kCodes + ws * kWBytes + row * 128;
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = *reinterpret_cast<const uint4*>(src + ((j ^ (row & 7)) << 4));
    };
    bool more = exists(it);
    if (more) {
      more = wait.warp(w_full(it % kW), (it / kW) & 1);
      if (more) read(it % kW);
    }
    while (more) {
      const int s = it % kStages;
      if (!wait.warp(empty(s), (it / kStages + 1) & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t h[16];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 v = c[2 * q + j];
          const int o = q >= 2 ? 4 : 0;  // the second 64 k: see the rows below
          widen(v.x, h[8 * j + o], h[8 * j + o + 1]);
          widen(v.y, h[8 * j + o + 2], h[8 * j + o + 3]);
          widen(v.z, h[8 * j + 4 - o], h[8 * j + 5 - o]);
          widen(v.w, h[8 * j + 6 - o], h[8 * j + 7 - o]);
        }
        __syncwarp();
        tmem_st16(tmem + lanes + kABase + s * kACols + q * 16, h);
      }
      // Only now: an arrival right behind the loads does not wait for them, and the
      // next codes came in before all lanes had read these (one run in 400).
      __syncwarp();
      if (lane == 0) mbar_arrive(w_empty(it % kW));
      it += 2;
      more = exists(it);
      const bool early = more && __all_sync(~0u, mbar_try(w_full(it % kW), (it / kW) & 1));
      if (early) read(it % kW);
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_leader(full(s));
      if (more && !early) {
        if (!wait.warp(w_full(it % kW), (it / kW) & 1)) break;
        read(it % kW);
      }
    }
  } else if (warp < 20) {
    // Rows to fp16 in shared memory, warps 12-15 the even stages and 16-19 the
    // odd ones.  Eight threads take the 128 codes of a row; a thread has rows
    // tid/8 + 16i and loads them a stage ahead of its need (two or more were no
    // faster: 4.20 ms for the prefill's product either way).
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    constexpr int RI = kRowsCta / 16;
    const int tid = threadIdx.x & 127, r_in = tid >> 3, kc = tid & 7;
    const uint32_t parity = (warp - 12) >> 2;
    int src[RI];
    int live = 0;            // rows of this CTA in the tile, a multiple of 16
    uint32_t it = parity;    // of all stages of this CTA's tiles
    uint32_t begin = 0, end = 0;  // stages of the present tile
    uint4 v[RI];
    auto fetch = [&]() -> bool {
      if (it >= end) {
        while (it >= end) {
          if (!cur.next(tile)) return false;
          begin = end;
          end += k_stages;
        }
        live = (tile.rows + 31) / 32 * 16;
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const int r = r_in + 16 * i, j = static_cast<int>(rank) * live + r;
          src[i] = r < live && j < tile.rows ? source_row(d, tile.r0 + j) : -1;
        }
      }
      const int k = static_cast<int>(it - begin) * kStageK + 16 * kc;
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        const int8_t* p = d.a + static_cast<int64_t>(src[i]) * d.K + k;
        if (k < d.K && src[i] >= 0) v[i] = ld_codes(p);
        if (kc == 0 && k + kAhead < d.K && src[i] >= 0) prefetch_line(p + kAhead);
      }
      return true;
    };
    // A thread's 16 codes fill two 16-byte pieces.  In the second 64 k they
    // change places (and the weights' with them: the order of k is free), so
    // that the eight threads of a row always store to eight groups of banks.
    const int first = (kc & 3) * 2 + (kc >> 2), second = first ^ 1;
    while (fetch()) {
      const int s = it % kStages;
      if (!wait.warp(empty(s), (it / kStages + 1) & 1)) break;
      uint8_t* half = smem + L::kB + s * kBBytes + (kc >> 2) * kHalf + r_in * 128;
      const int swizzle = r_in & 7;  // of row r_in + 16i too
      uint8_t* to0 = half + ((first ^ swizzle) << 4);
      uint8_t* to1 = half + ((second ^ swizzle) << 4);
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        if (r_in + 16 * i >= live) break;
        uint4 x, y;
        widen(v[i].x, x.x, x.y);
        widen(v[i].y, x.z, x.w);
        widen(v[i].z, y.x, y.y);
        widen(v[i].w, y.z, y.w);
        *reinterpret_cast<uint4*>(to0 + i * 16 * 128) = x;
        *reinterpret_cast<uint4*>(to1 + i * 16 * 128) = y;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        release_shared();
        mbar_arrive_leader(full(s));
      }
      it += 2;
    }
  } else {
    // scale, round, store: a thread has one channel and half the rows, warps
    // 20-23 the first half (in 32s) and 24-27 the other
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    float* sc = reinterpret_cast<float*>(smem + L::kScale) + (warp - 20) * kRowsCta;
    uint32_t* zr = reinterpret_cast<uint32_t*>(smem + L::kZero) + (warp - 20) * (kRowsCta / 32);
    uint32_t nt = 0;
    while (cur.next(tile)) {
      const int half = (tile.rows + 63) / 64 * 32;
      const int first = warp < 24 ? 0 : half;
      const int rows = warp < 24 ? min(half, tile.rows) : tile.rows - half;  // none, or less than none, are possible
      __syncwarp();
      for (int j = lane; j < kRowsCta; j += 32) {
        float v = 0.0f;
        bool zero = false;
        if (j < rows) {
          const int r = tile.r0 + first + j;
          const int s = d.rows ? d.rows[r] : r;
          zero = s < 0 || s >= d.a_rows;
          if (s >= d.a_rows) atomicOr(d.status, kStCapacity);
          if (!zero) v = d.a_scale[s];
        }
        sc[j] = v;
        const uint32_t m = __ballot_sync(~0u, zero);
        if (lane == 0) zr[j >> 5] = m;
      }
      __syncwarp();
      const int ch = tile.n0 + static_cast<int>(rank) * kChannels + (threadIdx.x & 127);
      const float ws = ch < d.N ? d.w_scale[static_cast<int64_t>(tile.e) * d.N + ch] : 0.0f;
      Out* out = static_cast<Out*>(d.out) + static_cast<int64_t>(tile.r0 + first) * d.N + ch;
      if (!wait.warp(d_full, nt & 1)) break;
      tc_fence_after();
      // 32 rows of the channel, scaled
      auto scaled = [&](int j0, float (&v)[32]) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld32(tmem + lanes + first + j0, r);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(sc + j0 + j);
          scale2(r[j], r[j + 1], f.x, f.y, ws, v[j], v[j + 1]);
          scale2(r[j + 2], r[j + 3], f.z, f.w, ws, v[j + 2], v[j + 3]);
        }
        const uint32_t zero = zr[j0 >> 5];
        if (zero != 0) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (zero >> j & 1) v[j] = 0.0f;
        }
      };
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_leader(d_empty);
      };
      if constexpr (sizeof(Out) == 2) {
        // The tile is held rounded in registers, so that the next one's
        // products may start before this one's stores.
        uint32_t y[kRowsCta / 2];
#pragma unroll
        for (int c = 0; c < kRowsCta / 32; ++c) {
          if (32 * c < rows) {
            float v[32];
            scaled(32 * c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[16 * c + j] = pack2(v[2 * j], v[2 * j + 1]);
          }
        }
        release();
        if (ch < d.N) {
          uint16_t* to = reinterpret_cast<uint16_t*>(out);
#pragma unroll
          for (int j = 0; j < kRowsCta / 2; ++j) {
            if (2 * j < rows) *to = static_cast<uint16_t>(y[j]);
            to += d.N;
            if (2 * j + 1 < rows) *to = static_cast<uint16_t>(y[j] >> 16);
            to += d.N;
          }
        }
      } else {
        for (int j0 = 0; j0 < rows; j0 += 32) {
          float v[32];
          scaled(j0, v);
          if (ch < d.N) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j0 + j < rows) out[static_cast<int64_t>(j0 + j) * d.N] = v[j];
          }
        }
        release();
      }
      ++nt;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_free<2>(tmem);
}

// ---- few rows per expert ----
//
// With few rows the weights' stream is what counts, and the layout above
// holds it back: a product whose A operand lies in tensor memory takes about
// 128 clocks however few columns it has, so 128 channels a CTA cannot be
// widened and multiplied as fast as they arrive.  Here the roles are
// exchanged: up to 128 rows are the A operand in tensor memory (lanes without
// a row cost nothing and are never read), 256 channels the B operand, widened
// in shared memory.  Per 16 steps of k shared memory moves 24 KB for 4096
// weights, 192 clocks, against 178 clocks at this GPU's memory bandwidth.
//
// With too few tiles for all SMs a cluster of S CTAs shares a tile along k; the
// partial sums meet in shared memory, each CTA finishing 256/S channels, and
// are added in the order of the CTAs.

constexpr int kNarrowThreads = 768;
constexpr int kNarrowRows = 128, kNarrowCh = 256;
// Mean rows per expert up to which this kernel is the faster one (many experts
// then need one row tile, some two): 64 experts, 7168 -> 4096, at 112 rows 460 us
// against the pairs' 487, at 120 466 against 489, at 128 583 against 493.  (2048 ->
// 7168 crosses earlier: at 96 rows 245 us against 276, at 120 296 against 282.)  One
// matrix: all of a tile.  And wherever its tiles are so few that two CTAs or more
// can share each along k: one matrix of 7168 -> 4096 at 256 rows 31.8 us against 53.4,
// at 512 42.1 against 54.4, at 768, which leaves a CTA a tile, 66.7 against 54.4.
constexpr int kNarrowMean = 120;
constexpr int kNW = 3;                       // stages of weight codes, 256 channels x 128 k
constexpr int kNS = 3;                       // widened stages, 64 k
constexpr int kNWBytes = kNarrowCh * 128;
constexpr int kNBBytes = kNarrowCh * 128;    // 64 halves a channel

struct NarrowShape {
  static constexpr int kW = 0, kB = kNW * kNWBytes;
  static constexpr int kScale = kB + kNS * kNBBytes;  // [4][256] channel scales, for each storing warp its own
  static constexpr int kRow = kScale + 4 * kNarrowCh * 4;  // [128] row scales and [128] zero rows (a shared tile's)
  static constexpr int kBars = kRow + 2 * kNarrowRows * 4;
  static constexpr int kNumBars = 2 * kNW + 2 * kNS + 3;
  static constexpr int kMisc = kBars + kNumBars * 8;  // kNumBars is odd: 8 bytes short of 16
  static constexpr int kGroups = kMisc + 16;
  static size_t bytes(int E) { return 1024 + kGroups + Groups::bytes(E); }
};

template <typename Out>
__device__ __forceinline__ void store16(Out* to, const float (&v)[16], int n, bool vec);
template <>
__device__ __forceinline__ void store16<float>(float* to, const float (&v)[16], int n, bool vec) {
  if (vec && n >= 16) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < n) to[j] = v[j];
  }
}
__device__ __forceinline__ void store16_packed(__nv_bfloat16* to, const uint32_t* y, int n, bool vec) {
  if (vec && n >= 16) {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(y[4], y[5], y[6], y[7]);
  } else {
    uint16_t* t = reinterpret_cast<uint16_t*>(to);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (2 * j < n) t[2 * j] = static_cast<uint16_t>(y[j]);
      if (2 * j + 1 < n) t[2 * j + 1] = static_cast<uint16_t>(y[j] >> 16);
    }
  }
}
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* to, const float (&v)[16], int n, bool vec) {
  uint32_t y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = pack2(v[2 * j], v[2 * j + 1]);
  store16_packed(to, y, n, vec);
}

template <typename Out>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    ep_matmul_narrow_kernel(const __grid_constant__ CUtensorMap wmap, MatmulDev d) {
  using L = NarrowShape;
  extern __shared__ uint8_t raw[];
  const uint32_t raw_at = smem_u32(raw);
  uint8_t* smem = raw + ((1024 - (raw_at & 1023)) & 1023);
  const uint32_t at = smem_u32(smem);
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  uint32_t rank, S;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(S));

  const uint32_t bars = at + L::kBars;
  auto w_full = [&](int s) { return bars + 8 * s; };
  auto w_empty = [&](int s) { return bars + 8 * (kNW + s); };
  auto full = [&](int s) { return bars + 8 * (2 * kNW + s); };
  auto empty = [&](int s) { return bars + 8 * (2 * kNW + kNS + s); };
  const uint32_t d_full = bars + 8 * (2 * kNW + 2 * kNS), d_empty = d_full + 8, drained = d_full + 16;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  const Groups groups(smem + L::kGroups, d.E);
  const Waiter wait{d.status, reinterpret_cast<volatile int*>(misc + 1), d.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNW; ++s) {
      mbar_init(w_full(s), 1);
      mbar_init(w_empty(s), 8);
    }
    for (int s = 0; s < kNS; ++s) {
      mbar_init(full(s), 8);
      mbar_init(empty(s), 1);
    }
    mbar_init(d_full, 1);
    mbar_init(d_empty, 4);
    mbar_init(drained, 1);
    misc[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<1>(at + L::kMisc);
  pdl_wait();
  if (warp == 2) find_groups(d, groups, kNarrowRows, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int units = (d.K + 127) / 128;  // of 128 k; this CTA's are [u0, u1)
  const int u0 = static_cast<int>(units * rank / S), u1 = static_cast<int>(units * (rank + 1) / S);
  const int k_end = min(d.K, u1 * 128);
  const int k_stages = (k_end - u0 * 128 + 63) / 64;
  Tile tile;
  tile.rows = 0;
  Cursor<kNarrowRows, kNarrowCh> cur(d, groups, blockIdx.x / S, gridDim.x / S);

  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int r = (warp & 3) * 32 + lane;
  float* sc = reinterpret_cast<float*>(smem + L::kScale) + (warp & 3) * kNarrowCh;
  float* row_scale = reinterpret_cast<float*>(smem + L::kRow);
  int* row_zero = reinterpret_cast<int*>(smem + L::kRow) + kNarrowRows;
  const bool vec = d.N % 8 == 0;
  float as = 0.0f;
  bool zero = true;
  auto scaled = [&](float (&v)[16], int c0) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 f = *reinterpret_cast<const float4*>(sc + c0 + j);
      v[j] = zero ? 0.0f : v[j] * as * f.x;
      v[j + 1] = zero ? 0.0f : v[j + 1] * as * f.y;
      v[j + 2] = zero ? 0.0f : v[j + 2] * as * f.z;
      v[j + 3] = zero ? 0.0f : v[j + 3] * as * f.w;
    }
  };
  bool done = false;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0 && lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      while (ok && cur.next(tile)) {
        if (d.suppress && blockIdx.x == 0) break;
        for (int u = u0; u < u1; ++u, ++it) {
          const int s = it % kNW;
          if (!(ok = wait(w_empty(s), (it / kNW + 1) & 1))) break;
          mbar_expect(w_full(s), kNWBytes);
          tma_weights(at + L::kW + s * kNWBytes, &wmap, u * 128, tile.n0, tile.e, w_full(s));
        }
      }
      for (uint32_t i = it > kNW ? it - kNW : 0; i < it; ++i) wait.drain(w_full(i % kNW), (i / kNW) & 1);
    } else if (warp == 1 && lane == 0) {
      uint32_t it = 0, nt = 0;
      bool ok = true;
      while (ok && cur.next(tile)) {
        const int n = min(kNarrowCh, (d.N - tile.n0 + 15) / 16 * 16);
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kNarrowRows >> 4) << 24);
        if (!(ok = wait(d_empty, (nt + 1) & 1))) break;
        bool ready = false;
        for (int j = 0; j < k_stages; ++j, ++it) {
          const int s = it % kNS;
          if (!ready && !(ok = wait(full(s), (it / kNS) & 1))) break;
          tc_fence_after();
          const uint32_t b = b_desc_low(at + L::kB + s * kNBBytes), a = tmem + kNarrowCh + s * 32;
          const uint32_t next = (it + 1) % kNS, parity = ((it + 1) / kNS) & 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i == 3) ready = j + 1 < k_stages && mbar_try(full(next), parity);
            mma_f16<1>(tmem, a + i * 8, b_desc(b + i * 2), idesc, (j | i) != 0);
          }
          mma_commit<1>(empty(s));
        }
        if (!ok) break;
        mma_commit<1>(d_full);
        ++nt;
      }
      mma_commit<1>(drained);
      wait.drain(drained, 0);
    }
  } else if (warp < 12) {
    // Rows to fp16 in tensor memory, warps 4-7 the even stages and 8-11 the odd
    // ones.  Four lanes take the 64 codes of a row, lane t codes 16t .. 16t + 15,
    // eight rows at a time; stored as 16 rows x 256 bits each, words 4t + b of a
    // row end up at place 4b + t, and the weights' do too.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int g = lane >> 2, k_lane = (lane & 3) * 16, r0 = (warp & 3) * 32;
    uint32_t it = (warp - 4) >> 2, begin = 0, end = 0;  // stages of all tiles, of the present one
    const int8_t* from[4] = {};
    uint4 v[4];
    auto fetch = [&]() -> bool {
      if (it >= end) {
        while (it >= end) {
          if (!cur.next(tile)) return false;
          begin = end;
          end += k_stages;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = r0 + g + 8 * i;
          const int src = row < tile.rows ? source_row(d, tile.r0 + row) : -1;
          from[i] = src >= 0 ? d.a + static_cast<int64_t>(src) * d.K : nullptr;
        }
      }
      const int k = u0 * 128 + static_cast<int>(it - begin) * 64 + k_lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (k < k_end && from[i] != nullptr) v[i] = ld_codes(from[i] + k);
        if ((it - begin) % 2 == 0 && k_lane == 0 && k + kAhead < k_end && from[i] != nullptr)
          prefetch_line(from[i] + k + kAhead);
      }
      return true;
    };
    while (fetch()) {
      const int s = it % kNS;
      if (!wait.warp(empty(s), (it / kNS + 1) & 1)) break;
      tc_fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (r0 + 16 * half < tile.rows) {
          uint32_t x[16];
          const uint4 a = v[2 * half], b = v[2 * half + 1];
          widen(a.x, x[0], x[1]);
          widen(b.x, x[2], x[3]);
          widen(a.y, x[4], x[5]);
          widen(b.y, x[6], x[7]);
          widen(a.z, x[8], x[9]);
          widen(b.z, x[10], x[11]);
          widen(a.w, x[12], x[13]);
          widen(b.w, x[14], x[15]);
          __syncwarp();
          tmem_st16x256(tmem + lanes + (static_cast<uint32_t>(16 * half) << 16) + kNarrowCh + s * 32, x);
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(s));
      it += 2;
    }
  } else if (warp < 20) {
    // Weights to fp16 in shared memory, warps 12-15 the first 64 k of every 128
    // and 16-19 the second; a thread has channels tid and tid + 128.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int half = (warp - 12) >> 2, tid = threadIdx.x & 127;
    uint32_t it = 0, stage = 0;
    bool ok = true;
    while (ok && cur.next(tile)) {
      const int channels = d.N - tile.n0;
      for (int u = u0; u < u1; ++u, ++it) {
        const int ws = it % kNW;
        if (!(ok = wait.warp(w_full(ws), (it / kNW) & 1))) break;
        const int j = 2 * (u - u0) + half;
        if (j < k_stages) {
          const uint32_t g = stage + j;
          const int s = g % kNS;
          if (!(ok = wait.warp(empty(s), (g / kNS + 1) & 1))) break;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint8_t* src = smem + L::kW + ws * kNWBytes + (tid + 128 * p) * 128;
            uint8_t* to = smem + L::kB + s * kNBBytes + (tid + 128 * p) * 128;
            uint4 c[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              c[q] = *reinterpret_cast<const uint4*>(src + (((4 * half + q) ^ (tid & 7)) << 4));
            if ((tid & ~31) + 128 * p < channels) {
              // word b of every 16 codes: places 4b .. 4b + 3
              auto put = [&](int b, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
                uint4 x, y;
                widen(w0, x.x, x.y);
                widen(w1, x.z, x.w);
                widen(w2, y.x, y.y);
                widen(w3, y.z, y.w);
                *reinterpret_cast<uint4*>(to + (((2 * b) ^ (tid & 7)) << 4)) = x;
                *reinterpret_cast<uint4*>(to + (((2 * b + 1) ^ (tid & 7)) << 4)) = y;
              };
              put(0, c[0].x, c[1].x, c[2].x, c[3].x);
              put(1, c[0].y, c[1].y, c[2].y, c[3].y);
              put(2, c[0].z, c[1].z, c[2].z, c[3].z);
              put(3, c[0].w, c[1].w, c[2].w, c[3].w);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(full(s));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(w_empty(ws));  // the codes are widened, not just loaded
      }
      stage += k_stages;
    }
  } else {
    // scale, round, store: a thread has one row and all channels
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    uint32_t nt = 0;
    while (cur.next(tile)) {
      __syncwarp();
      for (int j = lane; j < kNarrowCh; j += 32)
        sc[j] = tile.n0 + j < d.N ? d.w_scale[static_cast<int64_t>(tile.e) * d.N + tile.n0 + j] : 0.0f;
      zero = true;
      if (r < tile.rows) {
        const int s = d.rows ? d.rows[tile.r0 + r] : tile.r0 + r;
        if (s >= d.a_rows) atomicOr(d.status, kStCapacity);
        zero = s < 0 || s >= d.a_rows;
        if (!zero) as = d.a_scale[s];
      }
      __syncwarp();
      done = wait.warp(d_full, nt & 1);
      if (!done) break;
      tc_fence_after();
      if (S > 1) {
        row_scale[r] = as;
        row_zero[r] = zero;
        break;
      }
      const int channels = d.N - tile.n0;
      Out* out = static_cast<Out*>(d.out) + static_cast<int64_t>(tile.r0 + r) * d.N + tile.n0;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty);
      };
      if ((warp & 3) * 32 >= tile.rows) {
        release();
      } else if constexpr (sizeof(Out) == 2) {
        uint32_t y[kNarrowCh / 2];
#pragma unroll
        for (int c = 0; c < kNarrowCh / 16; ++c) {
          if (16 * c < channels) {
            float v[16];
            __syncwarp();
            tmem_ld(tmem + lanes + 16 * c, v);
            scaled(v, 16 * c);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[8 * c + j] = pack2(v[2 * j], v[2 * j + 1]);
          }
        }
        release();
        if (r < tile.rows) {
#pragma unroll
          for (int c = 0; c < kNarrowCh / 16; ++c)
            if (16 * c < channels) store16_packed(out + 16 * c, y + 8 * c, channels - 16 * c, vec);
        }
      } else {
        for (int c = 0; 16 * c < min(channels, kNarrowCh); ++c) {
          float v[16];
          __syncwarp();
          tmem_ld(tmem + lanes + 16 * c, v);
          scaled(v, 16 * c);
          if (r < tile.rows) store16<Out>(out + 16 * c, v, channels - 16 * c, vec);
        }
        release();
      }
      ++nt;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (S > 1) {
    // Partial sums: [CTA][channel/4][row][4] in the shared memory of the CTA
    // that finishes the channels; every stage there is done with by now.  The
    // four warps of each quarter of tensor memory's lanes take the chunks of 16
    // channels in turn.
    const bool have = blockIdx.x / S < cur.all() && misc[1] == 0;
    cluster_sync();
    tc_fence_after();
    const int per = kNarrowCh / 16 / static_cast<int>(S);  // chunks a CTA finishes
    Tile t1;
    Cursor<kNarrowRows, kNarrowCh> one(d, groups, blockIdx.x / S, gridDim.x / S);
    const bool live = warp >= 4 && warp < 20 && have && one.next(t1) && (warp & 3) * 32 < t1.rows;
    const int channels = d.N - t1.n0;
    if (live) {
#pragma unroll
      for (int i = 0; i < kNarrowCh / 64; ++i) {
        const int c = (warp >> 2) - 1 + 4 * i;
        if (16 * c >= channels) break;
        float v[16];
        __syncwarp();
        tmem_ld(tmem + lanes + 16 * c, v);
        const int owner = c / per;
        uint32_t to;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(to)
                     : "r"(at + (((rank * per + (c - owner * per)) * 4) * kNarrowRows + r) * 16), "r"(owner));
        if (r < t1.rows) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + q * kNarrowRows * 16),
                         "f"(v[4 * q]), "f"(v[4 * q + 1]), "f"(v[4 * q + 2]), "f"(v[4 * q + 3])
                         : "memory");
        }
      }
    }
    __syncwarp();
    cluster_sync();
    if (live && r < t1.rows) {
      as = row_scale[r];
      zero = row_zero[r] != 0;
      for (int i = (warp >> 2) - 1; i < per; i += 4) {
        const int c = static_cast<int>(rank) * per + i;
        if (16 * c >= channels) break;
        float v[16] = {};
        for (uint32_t g = 0; g < S; ++g) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 f = *reinterpret_cast<const float4*>(smem + (((g * per + i) * 4 + q) * kNarrowRows + r) * 16);
            v[4 * q] += f.x;
            v[4 * q + 1] += f.y;
            v[4 * q + 2] += f.z;
            v[4 * q + 3] += f.w;
          }
        }
        scaled(v, 16 * c);
        store16<Out>(static_cast<Out*>(d.out) + static_cast<int64_t>(t1.r0 + r) * d.N + t1.n0 + 16 * c, v,
                     channels - 16 * c, vec);
      }
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_free<1>(tmem);
}

// ---- a handful of rows per expert ----
//
// One token, or a decoding step's few rows per expert: all time goes into the
// weights' stream and into latency.  A CTA takes 16 channels x up to 16 rows;
// its 8 warps split k, each multiplies 16 x 8 x 32 codes at a time in integers
// (mma.sync s8: 157 TOP/s on this GPU, enough for 8 rows at its memory
// bandwidth, 16 at three quarters of it) straight from registers, and the
// integer sums meet in shared memory, exact in any order.  Operands come in
// 16-byte pieces as they lie in memory: the order of k inside a product is
// free as long as both operands agree, so lane t of a row takes k = 16t ..
// 16t + 15 of every 64.

// Measured (cold caches): four CTAs per SM with a unit of 128 k in flight each,
// 64 tokens top-6 over 64 experts 355 us (5.3 TB/s; 328 since weights are brought
// to L2 ahead); three with two units 421, five 380 us, 32 channels a CTA 355 us
// but 13.4 instead of 11.4 us for one token through one matrix.
constexpr int kThinRows = 16, kThinCh = 16, kThinWarps = 8;
// Mean rows per expert up to which this kernel is the faster one: 64 experts,
// 7168 -> 4096, at 6.8 rows 340 us against 351, at 7.5 348 against 351, at 8 357
// against 352.  (K = 2048 crosses earlier: 64 experts, 2048 -> 7168, at 6 rows 217 us
// against 204; 256 experts, 2048 -> 4096, at 6 rows 507 against 433.)
constexpr int kThinMean = 7;
// One matrix: up to so many rows, and products in all.  2048 -> 7168 at 32 rows
// 17.6 us against 19.6, at 64 23.7 against 19.6; 7168 -> 4096 at 32 24.7 against 33.9;
// 7168 -> 18432 at 8 38.1 against 42.1, at 9 46.2 against 42.1.
constexpr int kThinOneRows = 32;
constexpr int64_t kThinOneProducts = 1100000000;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights past L1.  A plan's weights are read once each: 8 tokens top-6 175 us,
// 181 through L1; one matrix that stays in L2 wants L1 (1 token, 2048 -> 7168,
// back to back: 6.3 us, 8.3 past it).
template <bool ONCE>
__device__ __forceinline__ uint4 ld_weights(const int8_t* p) {
  if (!ONCE) return ld_codes(p);
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// TILES: groups of 8 rows.  One warp's part of k: units [u0, u1) of 128 k.
// ahead: the channel whose weights this lane brings to L2 two units early (half
// the warp has one): 64 tokens top-6 339 -> 328 us, one token 37 -> 29 in a row;
// one unit early 335 us, three 335.
template <int TILES, bool ONCE>
__device__ __forceinline__ void thin_products(const int8_t* ahead, const int8_t* w0, const int8_t* w1,
                                              const int8_t* const (&x)[2], int u0, int u1, int k_lane, int K, int (&c)[2][4]) {
#pragma unroll 1
  for (int u = u0; u < u1; ++u) {
    if (ONCE && ahead != nullptr && u + 2 < u1) prefetch_line(ahead + (u + 2) * 128);
    uint4 a[2][2], b[TILES][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = u * 128 + h * 64 + k_lane;
      const bool in = k < K;
      const uint4 z = make_uint4(0, 0, 0, 0);
      a[0][h] = in ? ld_weights<ONCE>(w0 + k) : z;
      a[1][h] = in ? ld_weights<ONCE>(w1 + k) : z;
#pragma unroll
      for (int i = 0; i < TILES; ++i) b[i][h] = in && x[i] != nullptr ? ld_codes(x[i] + k) : z;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < TILES; ++i) {
        mma_s8(c[i], a[0][h].x, a[1][h].x, a[0][h].y, a[1][h].y, b[i][h].x, b[i][h].y);
        mma_s8(c[i], a[0][h].z, a[1][h].z, a[0][h].w, a[1][h].w, b[i][h].z, b[i][h].w);
      }
  }
}

// GROUPED: rows grouped by offsets; otherwise one matrix for all rows.
template <bool GROUPED, typename Out>
__global__ void __launch_bounds__(32 * kThinWarps, 4) ep_matmul_thin_kernel(MatmulDev d) {
  __shared__ int s_sum[kThinWarps][kThinRows][kThinCh + 1];
  __shared__ int s_tile[3];               // expert, first row, rows
  __shared__ int s_scan[kThinWarps];
  __shared__ int s_src[kThinRows];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned nch = (d.N + kThinCh - 1) / kThinCh;
  const int want = static_cast<int>(blockIdx.x / nch), n0 = static_cast<int>(blockIdx.x % nch) * kThinCh;
  if (threadIdx.x == 0) s_tile[2] = 0;
  if (!GROUPED) {
    if (threadIdx.x == 0) {
      s_tile[0] = 0;
      s_tile[1] = want * kThinRows;
      s_tile[2] = min(kThinRows, static_cast<int>(d.out_rows) - want * kThinRows);
    }
  } else {
    // the row tile `want` of all experts', 256 experts at a time
    if (blockIdx.x == 0 && threadIdx.x == 0 && d.offsets[d.E] > d.out_rows) atomicOr(d.status, kStCapacity);
    int before = 0;
    for (int e0 = 0; e0 < d.E; e0 += 32 * kThinWarps) {
      const int e = e0 + static_cast<int>(threadIdx.x);
      int r0 = 0, r1 = 0;
      if (e < d.E) {
        r0 = clamp_row(d.offsets[e], d.out_rows);
        r1 = clamp_row(d.offsets[e + 1], d.out_rows);
      }
      const int tiles = r1 > r0 ? (r1 - r0 + kThinRows - 1) / kThinRows : 0;
      int upto = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += v;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = upto;
      __syncthreads();
      int all = 0;
#pragma unroll
      for (int i = 0; i < kThinWarps; ++i) {
        if (i < warp) upto += s_scan[i];
        all += s_scan[i];
      }
      upto += before;
      if (want >= upto - tiles && want < upto) {
        s_tile[0] = e;
        s_tile[1] = r0 + (want - (upto - tiles)) * kThinRows;
        s_tile[2] = min(kThinRows, r1 - s_tile[1]);
      }
      before += all;
      if (before > want) break;
    }
  }
  __syncthreads();
  const int e = s_tile[0], first = s_tile[1], rows = s_tile[2];
  if (rows <= 0) return;
  const int8_t* w = d.w + static_cast<int64_t>(e) * d.N * d.K;
  const int units = (d.K + 127) / 128;
  const int u0 = units * warp / kThinWarps, u1 = units * (warp + 1) / kThinWarps;
  const int8_t* ahead = w + static_cast<int64_t>(min(n0 + (lane & 15), d.N - 1)) * d.K;
  if (GROUPED && u0 + (lane >> 4) < u1)  // units u0 and u0 + 1, while the rows are found
    prefetch_line(ahead + (u0 + (lane >> 4)) * 128);
  if (lane >= 16) ahead = nullptr;
  const int g = lane >> 2, t = lane & 3;
  // rows of codes of this lane's two columns
  const int8_t* x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i;
    int s = -1;
    if (r < rows) {
      s = d.rows ? d.rows[first + r] : first + r;
      if (s >= d.a_rows) {
        if (warp == 0 && t == 0) atomicOr(d.status, kStCapacity);
        s = -1;
      }
    }
    if (warp == 0 && t == 0) s_src[r] = s;
    x[i] = s >= 0 ? d.a + static_cast<int64_t>(s) * d.K : nullptr;
  }
  const int8_t* w0 = w + static_cast<int64_t>(min(n0 + g, d.N - 1)) * d.K;
  const int8_t* w1 = w + static_cast<int64_t>(min(n0 + g + 8, d.N - 1)) * d.K;
  int c[2][4] = {};
  if (rows > 8)
    thin_products<2, GROUPED>(ahead, w0, w1, x, u0, u1, 16 * t, d.K, c);
  else
    thin_products<1, GROUPED>(ahead, w0, w1, x, u0, u1, 16 * t, d.K, c);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) s_sum[warp][8 * i + 2 * t + (q & 1)][g + 8 * (q >> 1)] = c[i][q];
  __syncthreads();
  // one output a thread
  const int r = threadIdx.x / kThinCh, ch = threadIdx.x % kThinCh, n = n0 + ch;
  if (r < rows && n < d.N) {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kThinWarps; ++i) sum += s_sum[i][r][ch];
    const int s = s_src[r];
    float y = 0.0f;
    if (s >= 0) y = static_cast<float>(sum) * d.a_scale[s] * d.w_scale[static_cast<int64_t>(e) * d.N + n];
    static_cast<Out*>(d.out)[static_cast<int64_t>(first + r) * d.N + n] = static_cast<Out>(y);
  }
}

// ---- launch ----

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// What is found out once is kept only once it was found: a failure is asked again.
EncodeFn encoder() {
  static std::atomic<void*> found;
  void* p = found.load(std::memory_order_relaxed);
  if (p == nullptr) {
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return nullptr;
    found.store(p, std::memory_order_relaxed);
  }
  return reinterpret_cast<EncodeFn>(p);
}

// A number found out once per device (0: not yet), such as a kernel's limit of
// shared memory, which belongs to the device it was raised on.
class PerDevice {
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices];  // zero-initialised (static storage)

 public:
  int get(int dev) const { return dev >= 0 && dev < kDevices ? known_[dev].load(std::memory_order_relaxed) : 0; }
  void set(int dev, int v) {
    if (dev >= 0 && dev < kDevices) known_[dev].store(v, std::memory_order_relaxed);
  }
};

template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

// Clusters of n CTAs; a start before the end of the kernel ahead only where
// the kernels wait for it.
void set_cluster(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], unsigned n) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = EP_USE_PDL ? 2 : 1;
}

template <typename Out>
cudaError_t launch_pair(const MatmulDev& d, const CUtensorMap& map, cudaStream_t stream) {
  auto kernel = ep_matmul_pair_kernel<Out>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = PairShape::bytes(d.E);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  set_cluster(cfg, attr, 2);
  // pairs that run at once, for any number of experts (a CTA has its SM to
  // itself): a GPC with an odd number of SMs leaves one out
  static PerDevice rooms;
  int room = rooms.get(dev);
  if (room == 0) {
    err = allow_smem(kernel, PairShape::bytes(EP_MAX_EXPERTS));
    if (err != cudaSuccess) return err;
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms() / 2 * 2));
    if (cudaOccupancyMaxActiveClusters(&room, kernel, &cfg) == cudaSuccess && room > 0)
      rooms.set(dev, room);
    else
      room = num_sms() / 2;
  }
  // at most one tile per pair: the row tiles are not known here, but not more than this
  const int64_t most = (d.N + 2 * kChannels - 1) / (2 * kChannels) * most_row_tiles(d.out_rows, d.E, kRowsPair);
  cfg.gridDim = dim3(static_cast<unsigned>((most < room ? most : room) * 2));
  return cudaLaunchKernelEx(&cfg, kernel, map, d);
}

// CTAs that share a tile at most: 7168 -> 4096 at 128 rows 29.8 us with four, 42.1 with
// two, 42.1 with eight (clusters of eight do not fill the GPU).
constexpr unsigned kMaxShare = 4;

// Tiles of the few-row kernel: not more than this.
int64_t narrow_tiles(const MatmulDev& d) {
  return most_row_tiles(d.out_rows, d.E, kNarrowRows) * ((d.N + kNarrowCh - 1) / kNarrowCh);
}

template <typename Out>
cudaError_t launch_narrow(const MatmulDev& d, const CUtensorMap& map, cudaStream_t stream) {
  auto kernel = ep_matmul_narrow_kernel<Out>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  static PerDevice allowed;
  if (allowed.get(dev) == 0) {
    err = allow_smem(kernel, NarrowShape::bytes(EP_MAX_EXPERTS));
    if (err != cudaSuccess) return err;
    allowed.set(dev, 1);
  }
  const int64_t most = narrow_tiles(d), sms = num_sms();
  // CTAs a tile: as many as fill the SMs, each with two units of 128 k at least
  unsigned S = 1;
  while (S < kMaxShare && most * S * 2 <= sms && (d.K + 127) / 128 >= static_cast<int>(4 * S)) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((most < sms || S > 1 ? most : sms) * S));
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = NarrowShape::bytes(d.E);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  set_cluster(cfg, attr, S);
  return cudaLaunchKernelEx(&cfg, kernel, map, d);
}

}  // namespace

cudaError_t launch_matmul(const MatmulDev& d, bool out_bf16, cudaStream_t stream) {
  const bool thin = d.E == 1 ? d.out_rows <= kThinOneRows && d.out_rows * d.N * d.K <= kThinOneProducts
                             : d.out_rows <= kThinMean * static_cast<int64_t>(d.E);
  if (thin) {
    const unsigned grid = static_cast<unsigned>(most_row_tiles(d.out_rows, d.E, kThinRows) * ((d.N + kThinCh - 1) / kThinCh));
    auto kernel = d.offsets ? (out_bf16 ? ep_matmul_thin_kernel<true, __nv_bfloat16> : ep_matmul_thin_kernel<true, float>)
                            : (out_bf16 ? ep_matmul_thin_kernel<false, __nv_bfloat16> : ep_matmul_thin_kernel<false, float>);
    return launch_pdl(kernel, grid, 32 * kThinWarps, stream, d);
  }
  EncodeFn encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const bool narrow = d.out_rows <= (d.E == 1 ? kNarrowRows : kNarrowMean * static_cast<int64_t>(d.E)) ||
                      2 * narrow_tiles(d) <= num_sms();
  CUtensorMap map;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d.K), static_cast<cuuint64_t>(d.N), static_cast<cuuint64_t>(d.E)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d.K), static_cast<cuuint64_t>(d.K) * d.N};
  const cuuint32_t box[3] = {kStageK, static_cast<cuuint32_t>(narrow ? kNarrowCh : kChannels), 1}, step[3] = {1, 1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(d.w), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  if (narrow)
    return out_bf16 ? launch_narrow<__nv_bfloat16>(d, map, stream) : launch_narrow<float>(d, map, stream);
  return out_bf16 ? launch_pair<__nv_bfloat16>(d, map, stream) : launch_pair<float>(d, map, stream);
}

}  // namespace ep
