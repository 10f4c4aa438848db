// Products of E4M3 matrices with one fp32 scale for each 128 along K (rows of
// A: 1 x 128; weights W: 128 x 128), dense or grouped by expert, sm_100a:
//
//   C[m, n] = sum_b sA[m, b] sW[n / 128, b] sum_{k in block b} A[m, k] W[n, k]
//
// The tensor cores sum one block of 128 (four tcgen05.mma kind::f8f6f4, fp32 in
// TMEM); the epilogue warps then promote it: they read the 128 x 256 partial
// sums from TMEM and add them, times sA sW, to fp32 accumulators in their
// registers, while the tensor cores sum the next block into the other half of
// TMEM. Rows are the M side, so that a thread owns one row: its scale is one
// register, and a 128-column tile half has one weight scale.
//
// Two epilogues behind the last block:
//   MATMUL  C times an optional factor per row, bf16 or fp32
//   SWIGLU  the tile is 128 columns of the gate product and the matching 128 of
//           the up product: H = SiLU(gate) * up, and the tile's 128 columns are
//           one block of H, which leaves as E4M3 codes and a scale
// Sources: jacopoparretti "Mixture of experts, token by token", "Memory"
// (DeepSeek-V3 ships FP8 weights); Zero to Frontier 13.1, "The MoE layer" (the
// SwiGLU expert) and "In PyTorch" (grouped products over the experts).
//
// Warp roles (384 threads): warp 0 TMA producer, warp 1 TMEM owner and MMA
// issuer, warp 3 brings the scales and the tile's place, four K blocks at a time,
// into a ring in shared memory, warps 4..11 epilogue (warp w reads TMEM lanes
// 32 (w % 4)..+31, the two warps of a quadrant take 64 columns of each half of
// the tile). The epilogue threads hold 128 accumulators and two pieces of 32
// partial sums, so the first warpgroup hands registers to them (setmaxnreg):
// 4 x 32 x 56 + 8 x 32 x 224 = 64512, the 384 x 168 at launch.
//
// The epilogue warps touch no global memory inside the K loop: with their scales
// loaded by themselves, the wait for a TMEM read also waited for those loads in
// some builds and not in others (4736 x 4096 x 8192: 157 to 242 us by chance).
//
// Bound. Many rows: the way round between the MMAs of a block (512 cycles) and
// the epilogue's reads of it, about 960 cycles a block with the tensor pipe 53%
// active: 4736 x 4096 x 8192 in 151 to 160 us as a single call (2.0 to 2.1
// PFLOP/s), 177 us back to back (1.8), when the power cap holds the clock at 1.5
// GHz. A library product without block scales runs into the same cap and makes 2.15
// PFLOP/s of it (147 us): the cycles are this kernel's own. 8 experts' gate and up
// over 8192 rows, 4096 -> 14336: 1240 us back to back. Few rows: HBM; the same
// experts over 64 rows 166 us in the layer, 5.7 TB/s, 0.86 of the measured copy.
// Not kept, as slower: CTA pairs (tcgen05 cta_group::2; 171 us where this form then
// took 150), four TMEM buffers of 128 columns (173), loading a block's first columns
// while the last block is added (169), a deeper ring for few rows (181 -> 189 us).
// The K loop's code is sensitive: the same source compiled in parallel pieces (nvcc
// -split-compile) varied by 10%; these figures are of the library's own build.
//
// Tiles of 128 rows never straddle two experts; rows of a tile behind its
// expert's last row are computed from whatever lies there and not stored (a
// row's sums depend on that row alone). A tile of few rows loads a smaller box
// of A, and warps whose 32 rows are all behind the end skip their arithmetic.
//
// SPLIT (few tiles): a cluster of S CTAs shares one tile, each sums a
// range of K blocks, and the partial sums are added in rank order through
// distributed shared memory (in the then idle operand ring): no workspace, no
// atomics, the same bits every time.
//
// Every wait is bounded; see tc_gemm.cuh for the protocol.
#pragma once
#include "fp8_block.cuh"
#include "tc2_gemm.cuh"

namespace moe {
namespace f8b {

enum { MATMUL = 0, SWIGLU = 1 };
constexpr int BM = 128, BN = 256;
constexpr int A_BYTES = BM * BLK, B_BYTES = BN * BLK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 4;
constexpr int RING_BYTES = STAGES * STAGE_BYTES;
constexpr int NUM_THREADS = 384, EPI_WARPS = 8, FIRST_EPI_WARP = 4;
constexpr int CTRL_REGS = 56, EPI_REGS = 224;
constexpr int A_BOXES = 3;  // tensor maps of A with boxes of 16, 64 and 128 rows
constexpr int BAR_BYTES = 256;
constexpr int SEG_BYTES = 4 * (tc::MAX_E + 1);
constexpr int GROUP = 4;         // K blocks whose scales travel together
constexpr int SCALE_SLOTS = 4;   // groups in flight
constexpr int NUM_BARS = 2 * STAGES + 5 + 2 * SCALE_SLOTS + 4;
static_assert(8 * NUM_BARS + 8 <= BAR_BYTES, "barriers, TMEM address, abort flag");
struct ScaleSlot {
  float a[GROUP][BM];            // the rows' scales
  float2 w[GROUP];               // the weight scales of the tile's two halves
  int e, nb, row0, valid;        // the tile, in its first group
  int far[4];                    // [0]: scales whose product may be no normal number
};
constexpr int MAX_BYTES = 2 * 2 * BM * 4;  // SWIGLU: row maxima of the two half tiles, double-buffered
constexpr int STAGING_BYTES = EPI_WARPS * 2048;  // 32 rows of 64 output bytes a warp
constexpr int SMEM_BYTES = 1024 + RING_BYTES + STAGING_BYTES + BAR_BYTES +
                           SCALE_SLOTS * (int)sizeof(ScaleSlot) + SEG_BYTES + MAX_BYTES;
static_assert(sizeof(ScaleSlot) % 16 == 0, "slots stay aligned");
constexpr int DUMP_LD = BN + 4;  // floats a row of the split's partial sums (16-byte phases apart)
static_assert(SMEM_BYTES <= 232448, "shared memory per block");
static_assert(BM * DUMP_LD * 4 <= RING_BYTES, "the partial sums fit the ring");
static_assert(128 * CTRL_REGS + 256 * EPI_REGS <= NUM_THREADS * 168, "register split");

struct Maps {
  CUtensorMap a[A_BOXES];  // [M][K] codes, boxes of 128 bytes x 16, 64, 128 rows
  CUtensorMap w0, w1;      // [E][N][K] codes, boxes of 128 bytes x 128 rows (SWIGLU: gate, up)
};

struct Params {
  // rows of each expert: offsets [E + 1] (consecutive runs of rows), or the
  // layer's segments (tile_start in 128-row tiles, counts, capacity); neither: dense
  const int32_t* offsets;
  const int32_t* tile_start;
  const int32_t* counts;
  int64_t cap;
  int E, M, N;
  int n_tiles, k_blocks, n_blocks;  // tiles along N, blocks of 128 along K and N
  int max_tiles;                    // that segments without overlaps can have
  const float* a_scale;             // [M][k_blocks]
  const float* w_scale0;            // [E][n_blocks][k_blocks]
  const float* w_scale1;
  const float* row_scale;           // MATMUL: factor per row, NULL = 1
  void* out;                        // MATMUL: C; SWIGLU: codes of H
  int64_t out_ld;                   // elements
  int out_f32;                      // MATMUL
  int out_vec;                      // rows of `out` are 16-byte aligned
  float* out_scale;                 // SWIGLU: [M][n_blocks]
  unsigned long long timeout_ns, drain_timeout_ns;
  int* call_err;
};

__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Wait for this thread's TMEM loads; the registers pass through, so that no use
// of them can be scheduled before.
__device__ __forceinline__ void wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// The same registers' values from here on (behind a wait above).
__device__ __forceinline__ void pass_regs(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
// acc[i] += m * r[i]. Single fused adds: packed pairs (fma.rn.f32x2) came with 30
// to 110 register moves a block that differed from build to build, and were
// slower in each (4736 x 4096 x 8192: 136 to 163 us, single ones 134).
__device__ __forceinline__ void promote32(float* acc, const uint32_t* r, float m) {
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = fmaf(m, __uint_as_float(r[i]), acc[i]);
}
// Scales of 2^-62 .. 2^62 have a product that is a normal number. In a group of K
// blocks with any other scale (flagged by the warp that fetches them) the product is
// taken as fp32 holds it, and outside the normal numbers as that of one scale times
// 2^64, or of both times 2^-64; the sums take the rest, 2^-64 or 2^128, first, and
// are exact through it: a nonzero one lies within 2^-18 .. 2^25. So a scaled sum that
// fp32 can hold comes out as it should, where the plain product would have lost bits
// to a subnormal, or made inf of a number and NaN of a zero. What still under- or
// overflows here does so in the scaled sum itself.
constexpr float NEAR_LO = 0x1p-62f, NEAR_HI = 0x1p62f;
// 64 columns of a warp's sums in TMEM times 2^-64 or 2^128 as a w asks for; returns
// the factor that is left. In TMEM, before the sums are read, so that the code that
// reads and adds them stays what it is. Without any of this 4736 x 4096 x 8192 takes
// 147 us and 8192 rows over 8 experts (14336 -> 4096) 496; this way 151 and 512, the
// corrections in registers instead 167 and 557, in a loop of their own 516 and 1710
// (128 accumulators through two paths spill).
__device__ __noinline__ float far_block(uint32_t tb, float a, float w) {
  float m = a * w, f = 1.f, g = 1.f;
  if (fabsf(m) < FLT_MIN) {
    const bool less = fabsf(a) < fabsf(w);  // the smaller is below 2^-63, or one is zero
    m = (less ? a : w) * 0x1p64f * (less ? w : a);
    f = 0x1p-64f;
  } else if (!(fabsf(m) <= FLT_MAX)) {
    m = a * 0x1p-64f * (w * 0x1p-64f);
    f = g = 0x1p64f;
  }
#pragma unroll 1
  for (int i = 0; i < 64; i += 8) {
    float r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7])
        : "r"(tb + i)
        : "memory");
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = r[j] * f * g;
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(tb + i),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
        : "memory");
  }
  return m;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Bounded wait for the phase with `parity` of barrier `bar`; false when another
// role has given up or timeout_ns have passed (recorded, and the abort flag
// raised). In line, unlike
// the one in tc_gemm.cuh: the epilogue warps wait with 128 accumulators in
// registers. (What spills is the adding loop of MATMUL with SPLIT, 128 bytes a
// thread for its 64 sums in flight.) The first test does not suspend the warp and
// the limit is checked before the next, so that a limit of nothing ends the
// first wait that is not over.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                            unsigned long long timeout_ns) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 0;; ++it) {
    if ((it & 15u) == 0u) {
      if (*abort_flag) return false;
      if (static_cast<uint64_t>(clock64() - t0) >= wait_cycles(timeout_ns)) {
        atomicOr(&g_dev_error, DEVERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
    if (tc::mbar_try_wait(bar, parity)) return true;
  }
}

// True in one lane of a converged warp. The issuing roles run with all lanes and
// elect one for the copies and MMAs alone: issued from a branch on the lane
// index, an MMA took 95 cycles to issue, and the issuer bounded the kernel.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0u;
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
}
__device__ __forceinline__ uint2 bf16x4(const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

struct Tile {
  int e, nb, row0, valid;
};

// What the arrays say of expert e, and from that its first row and rows, clamped
// so that any contents of the arrays stay inside [0, M).
__device__ __forceinline__ int2 segment_load(const Params& p, int e) {
  if (p.offsets != nullptr) return make_int2(p.offsets[e], p.offsets[e + 1]);
  if (p.tile_start != nullptr) return make_int2(p.tile_start[e], p.counts[e]);
  return make_int2(0, p.M);
}
__device__ __forceinline__ int2 segment_of(const Params& p, int2 raw) {
  int64_t b = raw.x, t = raw.y;
  if (p.offsets == nullptr && p.tile_start != nullptr) {
    b *= ROW_TILE;
    t = b + (p.cap >= 0 && t > p.cap ? p.cap : t);
  }
  b = b < 0 ? 0 : (b > p.M ? p.M : b);
  t = t < b ? b : (t > p.M ? p.M : t);
  return make_int2((int)b, (int)(t - b));
}

// Tile order: expert by expert; within an expert the row tiles are fastest, so
// CTAs running at the same time share weight tiles through L2. s_mt: first row
// tile of each expert.
// In two steps, locate and place, so that the loads in between can be in flight.
struct Place {
  int e, nb, mi;
  int2 raw;
};
__device__ __forceinline__ Place locate(int tile, const Params& p, const int32_t* s_mt) {
  const int q = tile / p.n_tiles;
  int lo = 0, hi = p.E - 1;  // last expert whose first row tile is at or before q
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_mt[mid] <= q) lo = mid; else hi = mid - 1;
  }
  const int me = s_mt[lo + 1] - s_mt[lo];
  const int in_e = tile - p.n_tiles * s_mt[lo];
  Place l;
  l.e = lo;
  l.nb = in_e / me;
  l.mi = in_e - l.nb * me;
  l.raw = segment_load(p, lo);
  return l;
}
__device__ __forceinline__ Tile place(const Place& l, const Params& p) {
  const int2 seg = segment_of(p, l.raw);
  Tile t;
  t.e = l.e;
  t.nb = l.nb;
  t.row0 = seg.x + l.mi * BM;
  t.valid = min(BM, seg.y - l.mi * BM);
  return t;
}

// A warp's 32 rows of 64 output bytes, from registers (lane = row, four 16-byte
// pieces) to global memory: through shared memory, so that a store instruction
// writes 64 consecutive bytes of eight rows instead of 16 of 32. Piece c of row
// r lies at c ^ (r / 2 % 4): conflict-free both ways. `rows` of the 32 and
// `bytes` of the 64 exist; es = bytes of an element; vec: every row's first byte
// is 16-byte aligned.
__device__ __forceinline__ void store_rows64(uint8_t* stage, int lane, const uint4* v, uint8_t* out,
                                             int64_t ld_bytes, int rows, int bytes, int es,
                                             bool vec) {
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((c ^ (lane >> 1)) & 3) * 16) = v[c];
  __syncwarp();
  if (vec && (bytes & 15) == 0) {
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2);
      if (r < rows && c * 16 < bytes)
        *reinterpret_cast<uint4*>(out + r * ld_bytes + c * 16) =
            *reinterpret_cast<const uint4*>(stage + r * 64 + ((c ^ (r >> 1)) & 3) * 16);
    }
  } else {
    for (int r = 0; r < rows; ++r)
      for (int b = lane * es; b < bytes; b += 32 * es) {
        const uint8_t* from = stage + r * 64 + (((b >> 4) ^ (r >> 1)) & 3) * 16 + (b & 15);
        if (es == 2)
          *reinterpret_cast<uint16_t*>(out + r * ld_bytes + b) =
              *reinterpret_cast<const uint16_t*>(from);
        else
          *reinterpret_cast<uint32_t*>(out + r * ld_bytes + b) =
              *reinterpret_cast<const uint32_t*>(from);
      }
  }
}

// 32 columns of a warp's rows (lane = row; c: their sums) times the row's factor.
__device__ __forceinline__ void store32(const Params& p, uint8_t* stage, int lane, int64_t row0,
                                        int rows, int col, const float* c, float f) {
  if (col >= p.N) return;
  const int n = min(32, p.N - col);
  if (p.out_f32) {
    uint8_t* o = reinterpret_cast<uint8_t*>(static_cast<float*>(p.out) + row0 * p.out_ld + col);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = f * c[16 * h + 4 * i + j];
        v[i] = Vec16<float>::pack(x);
      }
      if (n > 16 * h)
        store_rows64(stage, lane, v, o + 64 * h, p.out_ld * 4, rows, 4 * min(16, n - 16 * h), 4,
                     p.out_vec);
    }
  } else {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = f * c[8 * i + j];
      v[i] = Vec16<__nv_bfloat16>::pack(x);
    }
    store_rows64(stage, lane, v,
                 reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(p.out) + row0 * p.out_ld + col),
                 p.out_ld * 2, rows, 2 * n, 2, p.out_vec);
  }
}

template <int MODE, bool SPLIT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    gemm_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = tc::smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* staging = smem + RING_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + STAGING_BYTES);
  // bars: full[STAGES], empty[STAGES], tfull[2], tempty[2], done, sfull[SCALE_SLOTS],
  // sempty[SCALE_SLOTS], maxima[4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  ScaleSlot* slots = reinterpret_cast<ScaleSlot*>(staging + STAGING_BYTES + BAR_BYTES);
  int32_t* s_mt = reinterpret_cast<int32_t*>(slots + SCALE_SLOTS);
  float* s_max = reinterpret_cast<float*>(s_mt + tc::MAX_E + 1);

  // warp index as a warp-uniform value: what follows from it can live in uniform
  // registers, which tcgen05.mma and the TMA copies take their operands from
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t stage0 = tc::smem_addr(smem);
  const uint32_t bar0 = tc::smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 4);
  auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 5 + s); };
  auto sempty_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 5 + SCALE_SLOTS + s); };
  auto maxima_bar = [&](int quad) { return bar0 + 8u * (2 * STAGES + 5 + 2 * SCALE_SLOTS + quad); };
  uint32_t rank = 0, ranks = 1;  // SPLIT: in the cluster
  if (SPLIT) {
    rank = tc2::cluster_ctarank();
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(full_bar(s), 1);
      tc::mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(tfull_bar(a), 1);
      tc::mbar_init(tempty_bar(a), EPI_WARPS);
    }
    tc::mbar_init(done_bar, 1);
    for (int s = 0; s < SCALE_SLOTS; ++s) {
      tc::mbar_init(sfull_bar(s), 1);
      tc::mbar_init(sempty_bar(s), EPI_WARPS);
    }
    for (int q = 0; q < 4; ++q) tc::mbar_init(maxima_bar(q), 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int b = 0; b < A_BOXES; ++b) tc::prefetch_map(&maps.a[b]);
    tc::prefetch_map(&maps.w0);
    if (MODE == SWIGLU) tc::prefetch_map(&maps.w1);
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_addr(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 2) {  // exclusive scan of the experts' row tiles
    int run = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int len = e < p.E ? segment_of(p, segment_load(p, e)).y : 0;
      const int v = (len + BM - 1) / BM;
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      // Offsets that overlap (an expert has at most 2^24 tiles) must not overflow.
      constexpr int LIMIT = 1 << 30;
      if (e < p.E) s_mt[e] = min(LIMIT, run + incl - v);
      run = min(LIMIT, run + __shfl_sync(0xffffffffu, incl, 31));
    }
    if (lane == 0) s_mt[p.E] = run;
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // at most 2^30 by the host; what overlapping offsets ask for beyond is left out
  const int total = (int)min((long long)p.n_tiles * s_mt[p.E], (long long)p.max_tiles);
  const unsigned long long tmo = p.timeout_ns, drain_tmo = p.drain_timeout_ns;
  // SPLIT: one tile a cluster, this CTA's range of K blocks
  const int first = blockIdx.x / ranks, step = SPLIT ? total : (int)gridDim.x;
  const int kb0 = SPLIT ? (int)((long long)p.k_blocks * rank / ranks) : 0;
  const int kb1 = SPLIT ? (int)((long long)p.k_blocks * (rank + 1) / ranks) : p.k_blocks;
  auto wait_ctrl = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_inline(bar, parity, abort_flag, tmo)) != 0;
  };

  if (warp < FIRST_EPI_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      uint32_t issued = 0, last_par = 0, phase = 0;
      int stage = 0;
      bool ok = true;
      Place next{};
      if (first < total) next = locate(first, p, s_mt);
      for (int tile = first; ok && tile < total; tile += step) {
        const Tile t = place(next, p);
        const int box = t.valid <= 16 ? 0 : (t.valid <= 64 ? 1 : 2);
        const uint32_t bytes = (box == 0 ? 16 : (box == 1 ? 64 : 128)) * BLK + B_BYTES;
        const int n0 = MODE == SWIGLU ? t.nb * BLK : t.nb * BN;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait_ctrl(empty_bar(stage), phase ^ 1u);
          if (!ok) break;
          const uint32_t sa = stage0 + stage * STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES;
          const int x = kb * (BLK / 4);  // coordinates in 32-bit words along K
          if (elect_one()) {
            const uint32_t fb = full_bar(stage);
            tc::mbar_expect_tx(fb, bytes);
            tc::tma_load_3d(sa, &maps.a[box], fb, x, t.row0, 0);
            tc::tma_load_3d(sb, &maps.w0, fb, x, n0, t.e);
            tc::tma_load_3d(sb + B_BYTES / 2, MODE == SWIGLU ? &maps.w1 : &maps.w0, fb, x,
                            MODE == SWIGLU ? n0 : n0 + BLK, t.e);
          }
          __syncwarp();
          // the next tile is looked up behind this one's first copy, so that no copy
          // waits for the look-up's loads
          if (kb == kb0 && tile + step < total) next = locate(tile + step, p, s_mt);
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && lane == 0)  // let every copy of this warp land before the CTA exits
        for (int s = 0; s < STAGES; ++s)
          if ((issued >> s) & 1u)
            tc::wait_drain(full_bar(s), (last_par >> s) & 1u, abort_flag, drain_tmo);
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t IDESC = tc::make_idesc_e4m3(BM, BN);
      int stage = 0;
      uint32_t phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      for (int tile = first; ok && tile < total; tile += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait_ctrl(full_bar(stage), phase) && wait_ctrl(tempty_bar(acc), acc_phase ^ 1u);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t sa = stage0 + stage * STAGE_BYTES;
          const uint64_t ad = tc::sw128_kmajor_desc(sa);
          const uint64_t bd = tc::sw128_kmajor_desc(sa + A_BYTES);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 codes = 32 bytes = +2 in the address field
              tc::tc_mma_e4m3(tmem_base + acc * BN, ad + 2u * kk, bd + 2u * kk, IDESC,
                              kk != 0 ? 1u : 0u);
            tc::tc_commit(empty_bar(stage));
            tc::tc_commit(tfull_bar(acc));
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          acc ^= 1u;
          if (acc == 0u) acc_phase ^= 1u;
        }
      }
      if (elect_one()) {
        tc::tc_commit(done_bar);
        tc::wait_drain(done_bar, 0u, abort_flag, drain_tmo);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ---------------------------------------------------------- scales
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first; ok && tile < total; tile += step) {
        const Tile t = place(locate(tile, p, s_mt), p);
        const int b0 = MODE == SWIGLU ? t.nb : 2 * t.nb;
        const int b1 = MODE == SWIGLU ? t.nb : min(2 * t.nb + 1, p.n_blocks - 1);
        const float* w0 = p.w_scale0 + ((int64_t)t.e * p.n_blocks + b0) * p.k_blocks;
        const float* w1 = (MODE == SWIGLU ? p.w_scale1 : p.w_scale0) +
                          ((int64_t)t.e * p.n_blocks + b1) * p.k_blocks;
        const float* as = p.a_scale + (int64_t)t.row0 * p.k_blocks;
        for (int kb = kb0; kb < kb1; kb += GROUP) {
          float v[4][GROUP], w = 1.f;  // 1 where there is none
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < GROUP; ++k) {
              const int r = 32 * i + lane;
              v[i][k] = r < t.valid && kb + k < kb1 ? __ldg(as + (int64_t)r * p.k_blocks + kb + k)
                                                    : 1.f;
            }
          if (lane < 2 * GROUP && kb + (lane >> 1) < kb1)
            w = __ldg((lane & 1 ? w1 : w0) + kb + (lane >> 1));
          ok = wait_ctrl(sempty_bar(slot), phase ^ 1u);
          if (!ok) break;
          ScaleSlot& s = slots[slot];
          // Zeros and negative scales are taken for far ones, and handled as what they
          // are; a NaN is passed over, and gives NaN either way.
          float lo = w, hi = w;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < GROUP; ++k) {
              s.a[k][32 * i + lane] = v[i][k];
              lo = fminf(lo, v[i][k]);
              hi = fmaxf(hi, v[i][k]);
            }
          if (lane < 2 * GROUP) reinterpret_cast<float*>(s.w)[lane] = w;
          const bool far = __any_sync(0xffffffffu, lo < NEAR_LO || hi > NEAR_HI);
          if (lane == 0) {
            s.e = t.e; s.nb = t.nb; s.row0 = t.row0; s.valid = t.valid;
            s.far[0] = far;
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(sfull_bar(slot));
          if (++slot == SCALE_SLOTS) { slot = 0; phase ^= 1u; }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    const int quad = warp & 3, half = (warp - FIRST_EPI_WARP) >> 2;
    const int r_in_tile = quad * 32 + lane;
    uint8_t* stage = staging + (warp - FIRST_EPI_WARP) * 2048;
    uint32_t acc = 0, acc_phase = 0, mphase = 0, sphase = 0;
    int slot = 0;
    bool ok = true, ready = false, sready = false, far = false;
    for (int tile = first; tile < total; tile += step) {
      float c[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) c[i] = 0.f;
      Tile t{};
      bool work = false;  // warp-uniform
      for (int kb = kb0; kb < kb1; ++kb) {
        const int k = (kb - kb0) & (GROUP - 1);
        // Both barriers of this block were tested before the last block's sums
        // were added; only one that had not completed is waited for. So was `far`
        // read, the group's flag.
        if (k == 0) {
          if (!__all_sync(0xffffffffu, sready)) {
            ok = wait_inline(sfull_bar(slot), sphase, abort_flag, tmo);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            far = slots[slot].far[0] != 0;
          }
          if (kb == kb0) {
            t.e = slots[slot].e; t.nb = slots[slot].nb;
            t.row0 = slots[slot].row0; t.valid = slots[slot].valid;
            work = quad * 32 < t.valid;
          }
        }
        float sa = slots[slot].a[k][r_in_tile];
        float2 sw = slots[slot].w[k];
        const uint32_t tb =
            tmem_base + acc * BN + half * 64 + (static_cast<uint32_t>(quad * 32) << 16);
        if (!__all_sync(0xffffffffu, ready && !far)) {
          ok = wait_inline(tfull_bar(acc), acc_phase, abort_flag, tmo);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (far && work) {  // in a branch that is there for the wait
            tc::tc_fence_after();
            sw.x = far_block(tb, sa, sw.x);
            sw.y = far_block(tb + 128, sa, sw.y);
            sa = 1.f;
          }
        }
        uint32_t r0[32], r1[32];
        if (work) {
          tc::tc_fence_after();
          // two loads in flight, each refilled as soon as its registers are free:
          // a load takes about 160 cycles beside the MMAs' own TMEM traffic, and
          // one at a time they were what bounded the kernel
          ld32(tb, r0);
          ld32(tb + 32, r1);
          wait_ld(r0);
          pass_regs(r1);
          promote32(c, r0, sa * sw.x);
          ld32(tb + 128, r0);
          promote32(c + 32, r1, sa * sw.x);
          ld32(tb + 160, r1);
          wait_ld(r0);
          pass_regs(r1);
          tc::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tempty_bar(acc));
        acc ^= 1u;
        if (acc == 0u) acc_phase ^= 1u;
        if (k == GROUP - 1 || kb == kb1 - 1) {  // the group's scales have been read
          if (lane == 0) tc::mbar_arrive(sempty_bar(slot));
          if (++slot == SCALE_SLOTS) { slot = 0; sphase ^= 1u; }
          sready = mbar_test(sfull_bar(slot), sphase);
          if (sready) far = slots[slot].far[0] != 0;
        }
        ready = mbar_test(tfull_bar(acc), acc_phase);
        if (work) {
          promote32(c + 64, r0, sa * sw.y);
          promote32(c + 96, r1, sa * sw.y);
        }
      }
      if (!ok) break;
      const bool row_ok = r_in_tile < t.valid;
      const int64_t row = (int64_t)t.row0 + r_in_tile;
      if (SPLIT) {
        // leave the partial sums in the ring: its copies and MMAs are over
        if (row_ok) {
          float* d = reinterpret_cast<float*>(smem) + (size_t)r_in_tile * DUMP_LD + half * 64;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            reinterpret_cast<float4*>(d)[i] =
                make_float4(c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]);
            reinterpret_cast<float4*>(d + 128)[i] = make_float4(
                c[64 + 4 * i], c[64 + 4 * i + 1], c[64 + 4 * i + 2], c[64 + 4 * i + 3]);
          }
        }
      } else if (MODE == MATMUL) {
        if (work) {
          const float f = row_ok && p.row_scale != nullptr ? p.row_scale[row] : 1.f;
          const int col = t.nb * BN + half * 64, rows = min(32, t.valid - quad * 32);
          const int64_t r0 = (int64_t)t.row0 + quad * 32;
          store32(p, stage, lane, r0, rows, col, c, f);
          store32(p, stage, lane, r0, rows, col + 32, c + 32, f);
          store32(p, stage, lane, r0, rows, col + 128, c + 64, f);
          store32(p, stage, lane, r0, rows, col + 160, c + 96, f);
        }
      } else if (work) {
        const int col = t.nb * BLK + half * 64;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          c[i] = silu_f32(c[i]) * c[64 + i];
          if (col + i < p.N) m = max_nan(m, fabsf(c[i]));
        }
        // The quadrant's two warps exchange their maxima, in two buffers in turn: a
        // warp comes back to a buffer only after its partner has arrived for the
        // other one, so has read this one. A barrier of their own, with a limit: a
        // warp may finish up to two tiles of one K block that its partner gave up.
        float* mx = s_max + mphase * 2 * BM;
        mx[half * BM + r_in_tile] = m;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(maxima_bar(quad));
        ok = wait_inline(maxima_bar(quad), mphase, abort_flag, tmo);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        mphase ^= 1u;
        m = max_nan(m, mx[(half ^ 1) * BM + r_in_tile]);
        // rows behind the end hold anything: a scale of 1 keeps their lanes off the
        // division path, which the whole warp would walk with them (64 rows over 8
        // experts: 212 -> 182 us)
        const float s = row_ok ? block_scale(m) : 1.f;
        const Divisor d(s);
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = make_uint4(encode4(c + 16 * i, d), encode4(c + 16 * i + 4, d),
                            encode4(c + 16 * i + 8, d), encode4(c + 16 * i + 12, d));
        if (row_ok && half == 0) p.out_scale[row * p.n_blocks + t.nb] = s;
        if (col < p.N)  // N is a multiple of 16
          store_rows64(stage, lane, v,
                       static_cast<uint8_t*>(p.out) + ((int64_t)t.row0 + quad * 32) * p.out_ld + col,
                       p.out_ld, min(32, t.valid - quad * 32), min(64, p.N - col), 4, true);
      }
    }
  }

  if (SPLIT) {
    __syncthreads();
    tc2::cluster_sync();  // every rank's partial sums are in its ring
    if (warp >= FIRST_EPI_WARP && first < total && !*abort_flag) {
      const Tile t = place(locate(first, p, s_mt), p);
      const int w = warp - FIRST_EPI_WARP;
      // A warp takes four rows at a time, a lane four columns of each half of the
      // tile; the sums of two ranks are in flight at once and added in rank order.
      constexpr int R = 4;
      const int stride = (int)ranks * EPI_WARPS;
      for (int r0 = (int)rank + (int)ranks * w; r0 < t.valid; r0 += stride * R) {
        float4 lo[R], hi[R];
#pragma unroll
        for (int i = 0; i < R; ++i) lo[i] = hi[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t k = 0; k < ranks; k += 2) {
          float4 x[2][R], y[2][R];
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const int r = r0 + i * stride;
              x[kk][i] = y[kk][i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (k + kk < ranks && r < t.valid) {
                const uint32_t a =
                    tc2::mapa_shared(stage0 + (r * DUMP_LD + lane * 4) * 4, k + kk);
                x[kk][i] = ld_cluster_v4(a);
                y[kk][i] = ld_cluster_v4(a + 512);
              }
            }
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < R; ++i) {
              add4(lo[i], x[kk][i]);
              add4(hi[i], y[kk][i]);
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int r = r0 + i * stride;
          if (r >= t.valid) break;  // warp-uniform
          const int64_t row = (int64_t)t.row0 + r;
          if (MODE == MATMUL) {
            const float f = p.row_scale != nullptr ? p.row_scale[row] : 1.f;
            const float v[8] = {f * lo[i].x, f * lo[i].y, f * lo[i].z, f * lo[i].w,
                                f * hi[i].x, f * hi[i].y, f * hi[i].z, f * hi[i].w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int n = t.nb * BN + h * 128 + lane * 4;
              const int64_t o = row * p.out_ld + n;
              if (p.out_vec && n + 4 <= p.N) {
                if (p.out_f32)
                  *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) =
                      make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
                else
                  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) =
                      bf16x4(v + 4 * h);
              } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (n + c < p.N) {
                    if (p.out_f32) static_cast<float*>(p.out)[o + c] = v[4 * h + c];
                    else static_cast<__nv_bfloat16*>(p.out)[o + c] = __float2bfloat16_rn(v[4 * h + c]);
                  }
              }
            }
          } else {
            const float h[4] = {silu_f32(lo[i].x) * hi[i].x, silu_f32(lo[i].y) * hi[i].y,
                                silu_f32(lo[i].z) * hi[i].z, silu_f32(lo[i].w) * hi[i].w};
            const int col = t.nb * BLK + lane * 4;
            float m = 0.f;
            if (col < p.N)  // N is a multiple of 16
              m = max_nan(max_nan(fabsf(h[0]), fabsf(h[1])), max_nan(fabsf(h[2]), fabsf(h[3])));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float s = block_scale(m);
            if (col < p.N)
              *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * p.out_ld + col) =
                  encode4(h, Divisor(s));
            if (lane == 0) p.out_scale[row * p.n_blocks + t.nb] = s;
          }
        }
      }
    }
    tc2::cluster_sync();  // nobody reads this ring any more
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  tc::record_call_status(abort_flag, p.call_err);
  if (warp == 1) {
    __syncwarp();
    tc::tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace f8b
}  // namespace moe
