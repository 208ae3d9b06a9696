// Latent attention over a cache held in 4 bits (format: latent_fp4.cuh), on
// the 5th-generation tensor cores:
//   out[h] = sum_t softmax_t(sm_scale * q_h . c_t) c_t   over a token set S,
// S either the tokens of the row's selected blocks and its partial tail
// (spx_sparse_mla_attn_fp4), or every token the row sees
// (spx_latent_attn_fp4).
//
// Operands.  A cached row is c_t = 2^E_t c'_t, E_t its largest group exponent
// (or that of a row among its 8 neighbours, where all of them are within 4) and
// c'_t exact in fp16; a query head is q_h = 2^-s_h q'_h with max |q'_h| in
// [2^14, 2^15), exact in fp16 down to 2^-32 of that.  So
//   z_t = log2(e) sm_scale 2^-s_h 2^E_t (q'_h . c'_t) + E_t   (base 2),
//   P_t = 2^(z_t - R),  O = sum_t P_t c'_t,  l = sum_t P_t 2^-E_t,
//   out = O / l,  lse = (R + log2 l) ln 2.
// The running maximum is taken of z, the size of a token's contribution to O,
// not of the logit alone, so P fits fp16 (11 bits where bf16 has 8: the
// output's error is then its own rounding, not P's) whatever the rows'
// exponents; R is the maximum less 7, so P's subnormals begin 2^21 below the
// largest term, and the maximum is raised lazily (at most 2^15 in all).  l is
// a sum of unrounded fp32 values.
//
// Work.  A unit is 64 (row, head) pairs that share a token list: 64 heads of
// a row, or, with fewer heads, several rows of a sequence.  All units' lists,
// in tiles of 64 tokens, form one sequence of tiles that is cut into equal
// parts, one per CTA (one CTA per SM), whatever the lengths.  A CTA walks its
// part as segments of units; a segment that is not its whole unit leaves its
// part in the workspace, and k_attn_fp4_combine joins the parts.
//
// One CTA, 20 warps, which pass items (a segment's queries, its tiles) through
// three shared-memory slots of 64 KiB:
//   list warps (2): the blocks of a tile and their positions; they copy its
//     codes and scales (17 KiB, cp.async) into a slot as soon as it is free;
//   converters (8): a warp expands its 8 tokens where they lie, from 4 bits to
//     fp16 in the 128-byte-swizzle layout; they also bring the queries, which
//     the workers take on to TMEM;
//   QK warp: S = Q C^T, 32 tcgen05.mma (M = 64, N = 64, K = 16), A in TMEM;
//   PV warp: O += P C, 8 tcgen05.mma (M = 64, N = 256, K = 16, C read MN-major
//     from the same slot), which gives the slot back;
//   workers (8): softmax and output.  A warp has 16 pairs and 32 of a tile's
//     tokens, the two threads of lanes i and 16 + i a pair.
// An M = 64 product uses 16 lanes of each TMEM quarter, so both halves of the
// lanes are used: lanes 0-15 the queries (columns 0-255) and two buffers of S
// (256-383), lanes 16-31 O (0-511).
//
// What bounds it.  An M = 64 product runs at half the tensor rate (2,048 cycles
// a tile: 0.36 ms for four sequences of 0.5-1M tokens, where it takes 0.65); a
// tile's operand reads (1,130 wavefronts of 128 bytes: the queries in TMEM save
// 512), its expansion and copies (about 1,300) share one shared-memory port;
// and a slot's round (copy, expand, QK, softmax, PV: about 10,000 cycles with
// three in flight) sets the pace at 3,500 cycles a tile.  Where units are short,
// their joints count: the next unit's queries go to TMEM before the last one's
// output is read from it, so that its first products run meanwhile (1,024 units
// of 33 tiles: 497 us with the output first, 479 so).  Tried and slower: two
// slots and the queries in shared memory (4,200); the converters loading their
// own rows into registers (3,800); bulk copies of 1 KiB blocks (the copy
// engine takes 75 cycles each: 5,600); 16 warps with one list for all (5,000).
#include <atomic>

#include "latent_fp4.cuh"
#include "spx_device.cuh"
#include "spx_internal.h"
#include "spx_launch.cuh"
#include "spx_warp_wait.cuh"

namespace spx {

namespace {

constexpr int kWork = 256;       // worker threads (warps 0-7)
constexpr int kConvWarp0 = 8;    // converter warps 8-15
constexpr int kConvWarps = 8;
constexpr int kQkWarp = 16;      // MMA issue
constexpr int kPvWarp = 17;
constexpr int kListWarp = 18;    // warps 18 and 19: token lists, loads of codes and scales
constexpr int kThreads = 20 * 32;  // 96 registers a thread
constexpr int kTT = 64;          // tokens per tile
constexpr int kM = 64;           // (row, head) pairs per unit (MMA M)
constexpr int kOct = 8;          // tokens of a tile that a converter warp takes
static_assert(kOct * kConvWarps == kTT, "one group of 8 tokens a warp");
constexpr int kRegion = 64 * 128;         // [64 rows x 128 B] = 8 KiB
constexpr int kSlotBytes = 8 * kRegion;   // a tile (or the queries) in fp16: 64 KiB
constexpr int kSlots = 3;
constexpr int kPBytes = kRegion;          // [64 x 64 tokens] fp16, two buffers
constexpr int kSmemBytes = 1024 + kSlots * kSlotBytes + 2 * kPBytes;
// TMEM columns: in lanes 0-15 of each quarter the queries (two fp16 values a
// column) and the logits, in lanes 16-31 the output
constexpr int kColS = 256;
constexpr int kNear = 4;        // exponents of 8 rows that share one reference, at most apart
constexpr float kLazy = 8.f;   // the maximum is raised when exceeded by more
constexpr float kLift = 7.f;   // P = 2^(z - max + 7)
constexpr float kPartScale = 8192.f;  // 2^13: a part of O, at most 6 in magnitude, in fp16
constexpr int kMaxGrid = 160;  // CTAs (one per SM, at most)
constexpr int kPartHalfs = kM * kLatent;
constexpr uint32_t kIdescF16 = (1u << 4) | (static_cast<uint32_t>(kM >> 4) << 24);  // f16 A, B; f32 D
constexpr uint32_t kIdescPV = kIdescF16 | ((256u >> 3) << 17) | (1u << 16);  // B MN-major
static_assert(kSmemBytes + 6 * 1024 <= 232448, "shared memory budget");

struct KParams {
  const __nv_bfloat16* q;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t seq_tok;
  int64_t len_cap;
  const int32_t* idx;
  const int32_t* count;
  const int64_t* n_vis;
  int heads, per_seq;
  int units, groups;       // groups of 64 heads per row (dense: or rgs > 1)
  int rows_per_unit, rgs;  // rows of a unit; units per (sequence, head group)
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  int2* comb;      // [grid] (unit, CTAs it spans) of the split unit that begins in a CTA
  float4* part_ml; // [2 grid][64] (R, l, sum of the weights / kPartScale)
  __half* part_o;  // [2 grid][64][512] kPartScale O / sum of the weights
};

// A slot's item as the list warps describe it to the other roles.
struct __align__(16) TileMeta {
  int unit;
  int bits;           // tokens of the tile's part of the list (0..64), and flags
  uint32_t valid[2];  // a bit per token that has a row in the cache
};
// first, last tile of its segment; not a tile but its segment's queries
enum : int { kFirst = 256, kLast = 512, kQueries = 1024 };

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Barrier of the two worker warps that share TMEM lane quarter qd (ids 1-4).
// (Instructions with .aligned want the warp converged: every divergent piece
// of code before one ends with a __syncwarp.)
__device__ __forceinline__ void pair_sync(int qd) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(1 + qd) : "memory");
}
// 16-byte asynchronous copy to shared memory, zeros where `valid` is false; the
// second makes an mbarrier arrival of the thread's copies so far.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Asks `bytes` (a multiple of 16) from a 16-byte aligned address into L2.
__device__ __forceinline__ void l2_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// Pairs of fp32 values in one register pair (the paired instructions round each
// as the single ones do).
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return pack2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(x));
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ void workers_sync() {
  __syncwarp();
  asm volatile("bar.sync 5, %0;" ::"n"(kWork) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t* v) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// One tcgen05.mma of fp16 operands by the elected lane (`el`, from elect_lane)
// of a warp that runs this with all its lanes.  The descriptors come as their
// low words, which hold the address in 16-byte units, so that a batch of MMAs
// costs one addition per operand and step.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t el;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(el));
  return el;
}
template <uint32_t kHi>
__device__ __forceinline__ void umma_f16(uint32_t el, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %6};\n\t"
      "mov.b64 b, {%3, %6};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 e, %0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, p;\n\t}" ::"r"(el),
      "r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kHi)
      : "memory");
}
// The same with A in TMEM (M = 64: lanes 0-15 of each quarter, as D's at lane
// offset 0; eight columns per step of K = 16).  A at lane offset 16 is a
// misaligned address.
template <uint32_t kHi>
__device__ __forceinline__ void umma_f16_ta(uint32_t el, uint32_t d_tmem, uint32_t a_tmem,
                                            uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%3, %6};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 e, %0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %4, p;\n\t}" ::"r"(el),
      "r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kHi)
      : "memory");
}
// High descriptor words: 1024 bytes between 8-row groups, version, 128-byte
// swizzle; low words: the address, and the distance between 64-element groups
// along MN (in bits 16-29; unused when K-major).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 16 lanes x 32 columns.
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---- units --------------------------------------------------------------------
__device__ __forceinline__ int clamp_len(const KParams& p, int64_t row) {
  const int64_t n = p.n_vis[row];
  return static_cast<int>(n < 0 ? 0 : (n > p.len_cap ? p.len_cap : n));
}

// First row of unit u and its head group; rows u holds.
struct UnitRows {
  int row0, nrows, hg;
};
template <bool kSparse>
__device__ __forceinline__ UnitRows unit_rows(const KParams& p, int u) {
  UnitRows r;
  const int rest = u >> (p.groups - 1);  // one or two groups
  r.hg = u & (p.groups - 1);
  if (kSparse) {
    r.row0 = rest;
    r.nrows = 1;
  } else {
    const int s = p.rgs == 1 ? rest : rest / p.rgs, rg = rest - s * p.rgs;
    r.row0 = s * p.per_seq + rg * p.rows_per_unit;
    r.nrows = min(p.rows_per_unit, p.per_seq - rg * p.rows_per_unit);
  }
  return r;
}

struct Unit {
  int n, cnt, S;  // visible tokens, selected blocks, tokens in the list
};
template <bool kSparse>
__device__ __forceinline__ Unit load_unit(const KParams& p, int u) {
  Unit x;
  const UnitRows r = unit_rows<kSparse>(p, u);
  x.n = clamp_len(p, r.row0);
  if (kSparse) {
    const int c = p.count[r.row0];
    x.cnt = min(min(max(c, 0), kTopK), x.n >> 2);  // 4 tokens a block
    x.S = x.cnt * kPool + (x.n & (kPool - 1));
  } else {
    for (int i = 1; i < r.nrows; ++i) x.n = max(x.n, clamp_len(p, r.row0 + i));
    x.cnt = 0;
    x.S = x.n;
  }
  return x;
}
// A unit without tokens still has one tile: its rows' outputs are written.
__device__ __forceinline__ int tiles_of(int S) { return (max(S, 1) - 1) / kTT + 1; }

// The part of the tile sequence a CTA owns, as every thread learns it.
struct Part {
  int begin, end, quota;
  int u0, off0;  // unit of tile `begin`, its first tile
};

// Scans the units' tile counts (every thread of the block calls this).  The
// loops stay rolled: the code runs once, and each of its lines is fetched for
// that.
template <bool kSparse>
__device__ __forceinline__ Part plan_part(const KParams& p, int* scratch /* [kThreads / 32 + 2] */) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Part part;
  int sum = 0, first = 0;  // tiles of unit tid, kept for the scan
#pragma unroll 1
  for (int u = tid; u < p.units; u += kThreads) {
    const int t = tiles_of(load_unit<kSparse>(p, u).S);
    if (u == tid) first = t;
    sum += t;
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) scratch[warp] = sum;
  __syncthreads();
  const int total = __reduce_add_sync(0xffffffffu, lane < kWarps ? scratch[lane] : 0);
  __syncthreads();
  const int g = static_cast<int>(gridDim.x);
  part.quota = (total - 1) / g + 1;
  const int64_t begin = static_cast<int64_t>(part.quota) * blockIdx.x;
  part.begin = static_cast<int>(begin < total ? begin : total);
  part.end = min(part.begin + min(part.quota, total - part.begin), total);
  part.u0 = 0;
  part.off0 = 0;
  int base = 0;
#pragma unroll 1
  for (int b = 0; part.begin < total; b += kThreads) {  // uniform; ends where the unit is found
    const int u = b + tid;
    int t = 0;
    if (u < p.units) t = b == 0 ? first : tiles_of(load_unit<kSparse>(p, u).S);
    const int inc = warp_incl_scan(t);
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    const int ws = warp_incl_scan(lane < kWarps ? scratch[lane] : 0);
    const int before = __shfl_sync(0xffffffffu, ws, warp > 0 ? warp - 1 : 0);
    const int off = base + (warp > 0 ? before : 0) + inc - t;
    base += __shfl_sync(0xffffffffu, ws, kWarps - 1);
    if (t > 0 && off <= part.begin && part.begin - off < t) {
      scratch[kWarps] = u;
      scratch[kWarps + 1] = off;
    }
    __syncthreads();
    if (part.begin < base) {
      part.u0 = scratch[kWarps];
      part.off0 = scratch[kWarps + 1];
      break;
    }
  }
  return part;
}

// ---- queries ------------------------------------------------------------------
// The row of a (row, head) pair within its unit; hpr heads a row, 16 at least.
__device__ __forceinline__ int pair_row(int m, int hpr) {
  return (m >= hpr ? 1 : 0) + (m >= 2 * hpr ? 1 : 0) + (m >= 3 * hpr ? 1 : 0);
}

// Rows w, w + 8, .. of the unit's 64 query rows to a shared-memory slot as
// fp16, each scaled by a power of two; hs[m] is what a product with it is
// multiplied by.  (Two rows at a time in a rolled loop: it runs once a segment,
// and unrolled over eight rows its instruction fetches took longer than its
// loads.)
template <bool kSparse>
__device__ __forceinline__ void load_q(const KParams& p, int u, uint32_t slot, float* hs, int w) {
  const int lane = threadIdx.x & 31;
  const UnitRows r = unit_rows<kSparse>(p, u);
  const int hpr = min(p.heads, kM);  // heads of a row in the unit
  const uint4* src = reinterpret_cast<const uint4*>(
      p.q + (static_cast<int64_t>(r.row0) * p.heads + r.hg * kM) * kLatent);
  // pairs past this one are padding (rows of a unit follow each other in q)
  const int pairs = min(r.nrows * hpr, p.heads * r.nrows - r.hg * kM);
  auto fetch = [&](int m, uint4* v) {
    v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u);
    if (m < pairs) {
      v[0] = src[m * 64 + lane];
      v[1] = src[m * 64 + 32 + lane];
    }
  };
  uint4 v[2][2], nx[2][2];
  fetch(w, v[0]);
  fetch(w + kConvWarps, v[1]);
#pragma unroll 1
  for (int m0 = w; m0 < kM; m0 += 2 * kConvWarps) {
    fetch(m0 + 2 * kConvWarps, nx[0]);
    fetch(m0 + 3 * kConvWarps, nx[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = m0 + i * kConvWarps;
      const uint32_t mask = 0x7FFF7FFFu;
      uint32_t a = __vmaxu2(__vmaxu2(v[i][0].x & mask, v[i][0].y & mask),
                            __vmaxu2(v[i][0].z & mask, v[i][0].w & mask));
      a = __vmaxu2(a, __vmaxu2(__vmaxu2(v[i][1].x & mask, v[i][1].y & mask),
                               __vmaxu2(v[i][1].z & mask, v[i][1].w & mask)));
      const uint32_t big = __reduce_max_sync(0xffffffffu, max(a & 0xFFFFu, a >> 16));
      const int s = min(14 + 127 - static_cast<int>(big >> 7), 110);
      const float f = __int_as_float((127 + s) << 23);  // 2^s
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 x = v[i][half];
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[k] = h2_bits(__floats2half2_rn(__uint_as_float(in[k] << 16) * f,
                                           __uint_as_float(in[k] & 0xFFFF0000u) * f));
        const int piece = 32 * half + lane;
        sts128(slot + (piece >> 3) * kRegion + m * 128 + (((piece & 7) ^ (m & 7)) << 4), o[0], o[1],
               o[2], o[3]);
      }
      if (lane == 0) hs[m] = p.scale_log2 * __int_as_float((127 - s) << 23);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i][0] = nx[i][0];
      v[i][1] = nx[i][1];
    }
  }
}

// ---- the kernel -----------------------------------------------------------------
template <bool kSparse>
__global__ void __launch_bounds__(kThreads, 1) k_attn_fp4(const KParams p) {
  extern __shared__ uint8_t dyn[];
  const uint32_t slot_u = (smem_u32(dyn) + 1023) & ~1023u, p_u = slot_u + kSlots * kSlotBytes;
  __shared__ uint64_t bar_raw[kSlots];   // slots: codes and scales have landed
  __shared__ uint64_t bar_full[kSlots];  // converted
  __shared__ uint64_t bar_free[kSlots];  // given back
  __shared__ uint64_t bar_qk[2], bar_p[2], bar_pv[2];  // S(t), P(t), O of tile t & 1 ready
  __shared__ uint64_t bar_q, bar_drain;                // queries in TMEM; all MMAs done
  __shared__ TileMeta meta_s[kSlots];
  // 2^E and E of each group of 8 tokens, or (0, inf): its tokens have their own,
  // in tf_s and te_s
  __shared__ __align__(16) float2 oct_s[kSlots][kConvWarps];
  __shared__ __align__(16) float tf_s[kSlots][kTT], te_s[kSlots][kTT];
  __shared__ float hs_s[4][kM];                       // per segment, mod 4
  __shared__ float red_m[2][2][kM];
  __shared__ float2 red_l[2][kM];
  __shared__ int scratch[kThreads / 32 + 2];
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bar_raw[i], 65);  // the list warps' lanes, and the item's description
      mbar_init(&bar_full[i], kConvWarps);
      mbar_init(&bar_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_qk[i], 1);
      mbar_init(&bar_p[i], kWork / 32);
      mbar_init(&bar_pv[i], 1);
    }
    mbar_init(&bar_q, 1);
    mbar_init(&bar_drain, 2);
    abort_s = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();  // (the set-up above ran beside the end of the stream's last kernel)
  const Part part = plan_part<kSparse>(p, scratch);
  const int ntiles = part.end - part.begin;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  volatile int* const abort = &abort_s;
  bool ok = true;  // no wait of this lane gave up

  // The items that pass through the slots: for each segment its queries, then
  // its tiles.
  struct Slot {
    int i = 0;             // slot of the next item
    uint32_t parity = 0;   // of the slot's round
    __device__ void next() {
      if (++i == kSlots) {
        i = 0;
        parity ^= 1u;
      }
    }
  } slot;

  if (ntiles == 0) {
    if (tid == 0 && p.comb) p.comb[blockIdx.x] = make_int2(-1, 0);
  } else if (warp >= kConvWarp0 && warp < kQkWarp) {
    // ======================= converter warps ==================================
    // The raw rows of a warp's 8 tokens lie where their fp16 rows will: blocks
    // of 4 tokens (1 KiB of codes) in its 1 KiB of the regions 0 and 1, the
    // scales (128 B) in region 2.  Lane 4 r + g has row r, code groups g, g +
    // 4, ..; odd rows take the groups in pairs swapped (g + 4 first), so that
    // the eight lanes of a load phase meet different banks.
    const int w = warp - kConvWarp0;
    const int r8 = lane >> 2, g4 = lane & 3;
    const bool odd = (r8 & 1) != 0, swap = (g4 & 2) != 0;
    const uint32_t raw_off = w * 1024 + (r8 >> 2) * kRegion + (r8 & 3) * 256 + g4 * 16 + (odd ? 64 : 0);
    // Lanes with g4 >= 2 store a group's four 16-byte pieces in the order 2, 3,
    // 0, 1: the eight lanes of a store phase (two rows, four groups) then meet
    // eight different bank groups.
    const uint32_t out_off = (w * kOct + r8) * 128 + (g4 >> 1) * kRegion +
                             (((4 * (g4 & 1)) ^ r8 ^ (g4 & 2)) << 4) + (odd ? 2 * kRegion : 0);
    const uint32_t odd_back = odd ? 0u - 4 * kRegion : 0u;
    int seg = 0;  // segments begun
#pragma unroll 1
    for (int t = 0; t < ntiles;) {
      ok = __all_sync(0xffffffffu, warp_wait(ok, &bar_raw[slot.i], slot.parity, abort));
      if (!ok) break;
      const uint32_t base = slot_u + slot.i * kSlotBytes;
      const int bits = meta_s[slot.i].bits;
      if (bits & kQueries) {  // (the workers take them to TMEM)
        load_q<kSparse>(p, meta_s[slot.i].unit, base, hs_s[seg & 3], w);
        ++seg;
      } else {
        ++t;
        const bool valid = ((meta_s[slot.i].valid[w >> 2] >> (8 * (w & 3) + r8)) & 1u) != 0;
        uint32_t c[4][4], sw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)  // groups 4 (k ^ odd) + g4
          lds128(base + ((raw_off + 128 * (k >> 1)) ^ (64 * (k & 1))), c[k]);
        lds128(base + w * 1024 + 2 * kRegion + r8 * 16, sw);
        // the row's largest exponent byte but 255 (a NaN group): bytes + 1 mod
        // 256, a word of four per lane; the bytes' carries are the NaN groups
        const uint32_t mine = swap ? (g4 & 1 ? sw[3] : sw[2]) : (g4 & 1 ? sw[1] : sw[0]);
        const uint32_t lo1 = (mine & 0x00FF00FFu) + 0x00010001u;
        const uint32_t hi1 = ((mine >> 8) & 0x00FF00FFu) + 0x00010001u;
        const bool nan = ((lo1 | hi1) & 0x01000100u) != 0;
        uint32_t mx = __vmaxu2(lo1 & 0x00FF00FFu, hi1 & 0x00FF00FFu);
        mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));  // (the raw rows are read)
        // biased exponent of the row, kept where 2^E and 2^-E are normal
        const int eb = min(max(static_cast<int>(max(mx & 0xFFFFu, mx >> 16)) - 1, 1), 253);
        // The 8 rows share the largest of their exponents where none is further
        // than 4 below it (they are then still exact: 2^-1 2^-15 2^-4 is above
        // fp16's last bit, and P loses at most 4 of its 31 bits below the
        // largest term); otherwise each row has its own.
        const int top = __reduce_max_sync(0xffffffffu, valid ? eb : 1);
        const int low = __reduce_min_sync(0xffffffffu, valid ? (nan ? -kNear : eb) : top);
        const bool wide = top - low > kNear;
        const int ref = wide ? eb : top;
        if (wide) {
          // A NaN group is NaN in its row's own E, and any number in the products'
          // operand: a NaN there would reach the rows of the unit that do not see
          // it (their weight is 0).
          const bool row_nan = ((__ballot_sync(0xffffffffu, nan) >> (4 * r8)) & 0xFu) != 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) sw[k] &= ~__vcmpeq4(sw[k], 0x01010101u * kFp4NanByte);
          if (g4 == 0) {
            tf_s[slot.i][w * kOct + r8] = __int_as_float(ref << 23);
            te_s[slot.i][w * kOct + r8] =
                row_nan ? __int_as_float(0x7FFFFFFF) : static_cast<float>(ref - 127);
          }
        }
        if (lane == 0)
          oct_s[slot.i][w] = wide ? make_float2(0.f, INFINITY)
                                  : make_float2(__int_as_float(ref << 23), static_cast<float>(ref - 127));
        // tokens up to the next multiple of 16 take part in the products
        if (w * kOct < max(16, ((bits & 0xFF) + 15) & ~15)) {
          __syncwarp();
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i] = base + (out_off ^ (i << 4));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int b = static_cast<int>(((odd ? sw[k ^ 1] : sw[k]) >> (8 * g4)) & 0xFFu);
            // 2^(e - E) in fp16 (0 from 2^-25 down; where there is no token the
            // codes are zeros)
            const __half2 s2 = __half2half2(
                __float2half_rn(__int_as_float(max(127 + b - ref, 97) << 23)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t h[4];
              fp4x8_to_half2x4(swap ? c[k][i ^ 2] : c[k][i], h);
#pragma unroll
              for (int e = 0; e < 4; ++e) h[e] = h2_bits(__hmul2(*reinterpret_cast<__half2*>(&h[e]), s2));
              sts128(out[i] + (k & 1 ? odd_back : 0) + 2 * kRegion * k, h[0], h[1], h[2], h[3]);
            }
          }
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_full[slot.i]);
      slot.next();
    }
  } else if (warp == kQkWarp || warp == kPvWarp) {
    // ======================= MMA issue ========================================
    // One warp issues S = Q C^T, the other O += P C.  A whole warp runs its
    // loop and one elected lane issues, so the descriptors are warp-uniform.
    const uint32_t el = elect_lane();
    const uint32_t tm0 = __shfl_sync(0xffffffffu, tmem, 0);
    // A segment's first tile follows its queries, whose slot is not waited for
    // here: the workers give it back without these warps.
    bool fresh = true;
    if (warp == kQkWarp) {
      int seg = 0;  // segments begun
#pragma unroll 1
      for (int t = 0; t < ntiles; ++t, slot.next()) {
        if (fresh) {
          slot.next();
          ok = warp_wait(ok, &bar_q, seg & 1, abort);
          ++seg;
        }
        // S buffer t & 1 is free once the softmax of tile t-2 has read it
        if (t >= 2) ok = warp_wait(ok, &bar_p[t & 1], ((t - 2) >> 1) & 1, abort);
        ok = warp_wait(ok, &bar_full[slot.i], slot.parity, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int bits = meta_s[slot.i].bits;
        fresh = (bits & kLast) != 0;
        tc_fence_after();
        const uint32_t n16 = static_cast<uint32_t>(max(16, ((bits & 0xFF) + 15) & ~15));
        const uint32_t idesc = kIdescF16 | ((n16 >> 3) << 17);
        const uint32_t d = tm0 + kColS + 64 * (t & 1);
        const uint32_t k_lo = desc_lo(slot_u + slot.i * kSlotBytes, 16);
#pragma unroll 1
        for (int k = 0; k < kLatent / 64; ++k) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            umma_f16_ta<kDescHi>(el, d, tm0 + 32 * k + 8 * i, k_lo + ((k * kRegion + i * 32) >> 4),
                                 idesc, k + i > 0 ? 1u : 0u);
        }
        umma_commit_elect(&bar_qk[t & 1]);
      }
    } else {
#pragma unroll 1
      for (int t = 0; t < ntiles; ++t, slot.next()) {
        if (fresh) slot.next();
        ok = warp_wait(ok, &bar_full[slot.i], slot.parity, abort);
        const int bits = meta_s[slot.i].bits;
        fresh = (bits & kLast) != 0;
        const int ks = max(1, ((bits & 0xFF) + 15) >> 4);
        ok = warp_wait(ok, &bar_p[t & 1], (t >> 1) & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t p_lo = desc_lo(p_u + (t & 1) * kPBytes, 16);
        const uint32_t c_lo = desc_lo(slot_u + slot.i * kSlotBytes, kRegion);
#pragma unroll
        for (int nh = 0; nh < 2; ++nh) {
#pragma unroll
          for (int k = 0; k < kTT / 16; ++k)
            if (k < ks)
              umma_f16<kDescHi>(el, tm0 + (16u << 16) + 256 * nh, p_lo + (k * 32 >> 4),
                                c_lo + ((nh * 4 * kRegion + k * 16 * 128) >> 4), kIdescPV,
                                (!(bits & kFirst) || k > 0) ? 1u : 0u);
        }
        umma_commit_elect(&bar_pv[t & 1]);
        umma_commit_elect(&bar_free[slot.i]);
      }
    }
    // every MMA issued completes before TMEM is released
    umma_commit_elect(&bar_drain);
    {
      volatile int no_abort = 0;
      warp_wait(true, &bar_drain, 0, &no_abort);
    }
  } else if (warp >= kListWarp) {
    // ======================= list warps =======================================
    // Lane i < 16 finds block i of a tile (4 tokens of the list: a selected
    // block, the partial tail, or four tokens in a row); the warps copy the
    // blocks' codes and scales into the tile's slot as soon as that is free.
    // Block ids are read a tile ahead; a whole cache's rows are asked into L2 a
    // tile ahead.  (cp.async, not bulk copies: the copy engine takes about 75
    // cycles for each, and a tile would need 32.)
    const int lw = warp - kListWarp;  // even blocks, odd blocks
    int u = part.u0;
    Unit un = load_unit<kSparse>(p, u), nxt{};
    int t_org = part.off0 - part.begin;  // CTA tiles [t_org, t_end) are u's
    int t_end = t_org + tiles_of(un.S);
    int2 comb = make_int2(-1, 0);
    int64_t tok0;
    const int32_t* ids;
    auto enter_unit = [&] {
      if (u + 1 < p.units) nxt = load_unit<kSparse>(p, u + 1);
      const int row0 = unit_rows<kSparse>(p, u).row0;
      tok0 = static_cast<int64_t>(kSparse ? row0 : row0 / p.per_seq) * p.seq_tok;
      ids = p.idx + static_cast<int64_t>(row0) * kTopK;  // (unused when dense)
      if (lane == 0 && lw == 1 && t_end < ntiles) {  // the next unit's queries, into L2
        const UnitRows r = unit_rows<kSparse>(p, u + 1);
        l2_prefetch(p.q + (static_cast<int64_t>(r.row0) * p.heads + r.hg * kM) * kLatent,
                    min(r.nrows * min(p.heads, kM), p.heads * r.nrows - r.hg * kM) * kLatent * 2);
      }
      if (t_org >= 0 && t_end > ntiles)  // the split unit that begins here
        comb = make_int2(u, (part.begin + t_end - 1) / part.quota - static_cast<int>(blockIdx.x) + 1);
    };
    int pos = 0, nt = 0;  // of this lane's block: first token, tokens (0..4)
    int tok_t = 0;        // the tile's first list entry
    TileMeta m;
    auto request = [&](int t) {  // the blocks of tile t
      if (t >= t_end) {
        ++u;
        un = nxt;
        t_org = t_end;
        t_end = t_org + tiles_of(un.S);
        enter_unit();
      }
      tok_t = (t - t_org) * kTT;
      m.unit = u;
      m.bits = max(0, min(un.S - tok_t, kTT)) | (t == max(t_org, 0) ? kFirst : 0) |
               (t == min(t_end, ntiles) - 1 ? kLast : 0);
      const int j = tok_t + (lane & 15) * kPool;
      pos = j;
      nt = max(0, min(un.S - j, kPool));
      if (kSparse && nt > 0) {
        if (j < un.cnt * kPool) {
          const int b = ids[j >> 2];
          if (b < 0 || b >= un.n >> 2)
            nt = 0;
          else
            pos = b * kPool;
        } else {
          pos = un.n & ~(kPool - 1);
        }
      }
    };
    enter_unit();
    request(0);
    int round = 0;  // items passed, up to kSlots
    auto wait_free = [&] {
      if (round < kSlots)
        ++round;
      else
        ok = __all_sync(0xffffffffu, warp_wait(ok, &bar_free[slot.i], slot.parity ^ 1u, abort));
    };
    auto publish = [&](const TileMeta& x) {  // the item of the slot, by lane 0
      if (lane == 0 && lw == 0) {
        meta_s[slot.i] = x;
        mbar_arrive(&bar_raw[slot.i]);
      }
    };
#pragma unroll 1
    for (int t = 0; t < ntiles; ++t) {
      if (m.bits & kFirst) {
        wait_free();
        if (!ok) break;
        TileMeta x = m;
        x.bits = kQueries;
        publish(x);
        mbar_arrive(&bar_raw[slot.i]);
        slot.next();
      }
      wait_free();
      if (!ok) break;
      const uint32_t v = lane < 16 ? ((1u << nt) - 1u) << (4 * (lane & 7)) : 0u;
      m.valid[0] = __reduce_or_sync(0xffffffffu, lane < 8 ? v : 0u);
      m.valid[1] = __reduce_or_sync(0xffffffffu, lane < 8 ? 0u : v);
      publish(m);
      const uint32_t dst = slot_u + slot.i * kSlotBytes;
      const uint8_t* codes = p.codes + tok0 * kFp4CodeBytes + lane * 16;
      const int nblk = max(4, ((m.bits & 0xFF) + 15) / 16 * 4);  // a multiple of 16 tokens
#pragma unroll 4
      for (int i = lw; i < nblk; i += 2) {  // a block's 1 KiB: two copies a lane
        const int n_i = __shfl_sync(0xffffffffu, nt, i);
        const int at = __shfl_sync(0xffffffffu, pos, i);
        const uint32_t d = dst + (i >> 1) * 1024 + lw * kRegion + lane * 16;
        const uint8_t* src = codes + static_cast<int64_t>(at) * kFp4CodeBytes;
        const bool v0 = (lane >> 4) < n_i, v1 = 2 + (lane >> 4) < n_i;
        cp_async16(d, v0 ? src : p.codes, v0);
        cp_async16(d + 512, v1 ? src + 512 : p.codes, v1);
      }
      {  // scales of blocks 8 lw .. 8 lw + 7: a token's 16 bytes a lane
        const int i = 8 * lw + (lane >> 2), tk = lane & 3;
        const int n_i = __shfl_sync(0xffffffffu, nt, i), at = __shfl_sync(0xffffffffu, pos, i);
        cp_async16(dst + (i >> 1) * 1024 + 2 * kRegion + (i & 1) * 64 + tk * 16,
                   p.scales + (tk < n_i ? tok0 + at + tk : 0) * kFp4Groups, tk < n_i);
      }
      cp_async_arrive(&bar_raw[slot.i]);
      slot.next();
      if (t + 1 < ntiles) {
        request(t + 1);
        if (!kSparse && lane == 0 && lw == 1 && (m.bits & 0xFF) > 0) {
          const int64_t at = tok0 + tok_t;
          l2_prefetch(p.codes + at * kFp4CodeBytes, (m.bits & 0xFF) * kFp4CodeBytes);
          l2_prefetch(p.scales + at * kFp4Groups, (m.bits & 0xFF) * kFp4Groups);
        }
      }
    }
    if (lane == 0 && lw == 0 && p.comb) p.comb[blockIdx.x] = comb;
    asm volatile("cp.async.wait_all;" ::: "memory");  // nothing lands once the block is gone
  } else if (warp < kConvWarp0) {
    // ======================= workers ==========================================
    const int qd = warp & 3, th = warp >> 2, half = lane >> 4;
    const int m = qd * 16 + (lane & 15);  // this thread's (row, head) pair of the unit
    const uint32_t tm_q = tmem + (static_cast<uint32_t>(qd * 32) << 16);  // this lane quarter
    const int hpr = min(p.heads, kM);
    // The workers wait for one another at named barriers, which have no limit,
    // so what they pass must not depend on a wait that may have given up: the
    // segments' ends come from the units' lengths, not from the slots.
    int u = part.u0, t_org = part.off0 - part.begin;  // CTA tiles t_org .. are unit u's
    int seg = 0, seg_end = 0, tiles = 0, row_lim = 0;
    int64_t out_row = -1;  // row of out of this thread, or -1
    float hs = 0.f, m_run = -INFINITY, l_run = 0.f, w_run = 0.f;  // w_run: sum of the weights
    // A segment's queries, from their slot to TMEM: 16-lane stores, which leave O
    // in the other lanes alone, so that the segment's first products start while
    // the last one's output is still written.  (Thread 4 r + c of a 16 x 256-bit
    // store has columns 2 c, 2 c + 1 of rows r and r + 8.)
    auto take_queries = [&] {
      ok = warp_wait(ok, &bar_full[slot.i], slot.parity, abort);
      const float next_hs = hs_s[seg & 3][m];
      ++seg;
#pragma unroll 1
      for (int r = 4 * th; r < 4 * th + 4; ++r) {  // 64 dims: 32 columns
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = qd * 16 + (lane >> 2) + 8 * (i & 1), piece = (i & 6) + ((lane & 3) >> 1);
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                       : "=r"(v[2 * i]), "=r"(v[2 * i + 1])
                       : "r"(slot_u + slot.i * kSlotBytes + r * kRegion + row * 128 +
                             ((piece ^ (row & 7)) << 4) + 8 * (lane & 1))
                       : "memory");
        }
        tmem_st_16x256b_x4(tm_q + 32 * r, v);
      }
      tc_fence_before();
      workers_sync();  // every worker's part is there
      if (tid == 0) {
        mbar_arrive(&bar_q);
        mbar_arrive(&bar_free[slot.i]);
      }
      slot.next();
      return next_hs;
    };
    auto enter_segment = [&] {  // unit u's part of this CTA
      const Unit un = load_unit<kSparse>(p, u);
      tiles = tiles_of(un.S);
      seg_end = min(t_org + tiles, ntiles);
      m_run = -INFINITY;
      l_run = w_run = 0.f;
      const UnitRows ur = unit_rows<kSparse>(p, u);
      const int rr = pair_row(m, hpr), h = ur.hg * kM + m - rr * hpr;
      const bool mine = rr < ur.nrows && h < p.heads;
      out_row = mine ? static_cast<int64_t>(ur.row0 + rr) * p.heads + h : -1;
      // rows of one unit may see different numbers of tokens
      row_lim = !kSparse && p.rows_per_unit > 1 ? (mine ? clamp_len(p, ur.row0 + rr) : 0)
                                                : 0x7fffffff;
    };
    enter_segment();
    hs = take_queries();
#pragma unroll 1
    for (int t = 0; t < ntiles;) {
      const int buf = t & 1;
      ok = warp_wait(ok, &bar_full[slot.i], slot.parity, abort);
      // (2^E, E) of this thread's two groups of 8 tokens
      const uint32_t valid = meta_s[slot.i].valid[th];
      uint32_t oc[4];
      lds128(smem_u32(&oct_s[slot.i][4 * th + 2 * half]), oc);
      const bool own = __any_sync(0xffffffffu, oc[1] == 0x7F800000u || oc[3] == 0x7F800000u);
      const uint32_t tf_u = smem_u32(&tf_s[slot.i][32 * th + 16 * half]),
                     te_u = smem_u32(&te_s[slot.i][32 * th + 16 * half]);
      slot.next();
      // P buffer t & 1 is free once PV(t-2) is done
      if (t >= 2) ok = warp_wait(ok, &bar_pv[buf], ((t - 2) >> 1) & 1, abort);
      ok = warp_wait(ok, &bar_qk[buf], (t >> 1) & 1, abort);
      tc_fence_after();
      uint32_t z[16];  // (floats, in pairs for the paired instructions)
      {
        // lanes 0-15 receive the 32 logits of their head in this warp's half
        // of the tile; tokens 16-31 of it go to the partner lane
        uint32_t a[32];
        tmem_ld_x32_async(tm_q + kColS + 64 * buf + 32 * th, a);
        tmem_ld_wait_regs<32>(a);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t v = __shfl_xor_sync(0xffffffffu, a[16 + i], 16);
          z[i] = half ? v : a[i];
        }
      }
      auto factors = [&](int i, uint32_t* f, uint32_t* e) {  // of tokens i .. i + 3
        f[0] = f[1] = f[2] = f[3] = oc[i < 8 ? 0 : 2];
        e[0] = e[1] = e[2] = e[3] = oc[i < 8 ? 1 : 3];
        if (e[0] == 0x7F800000u) {
          lds128(tf_u + 4 * i, f);
          lds128(te_u + 4 * i, e);
        }
      };
      if (!own) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float f = __uint_as_float(oc[2 * g]) * hs, e = __uint_as_float(oc[2 * g + 1]);
#pragma unroll
          for (int i = 8 * g; i < 8 * g + 8; i += 2) {
            const float2 x = unpack2(fma2(pack2(z[i], z[i + 1]), pack2(f, f), pack2(e, e)));
            z[i] = __float_as_uint(x.x);
            z[i + 1] = __float_as_uint(x.y);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          uint32_t f[4], e[4];
          factors(i, f, e);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            z[i + k] = __float_as_uint(fmaf(__uint_as_float(z[i + k]), hs * __uint_as_float(f[k]),
                                            __uint_as_float(e[k])));
        }
      }
      {
        const int lim = row_lim - (t - t_org) * kTT - 32 * th - 16 * half;
        uint32_t sees = (valid >> (16 * half)) & 0xFFFFu;
        if (lim < 16) sees &= (1u << max(lim, 0)) - 1u;
        if (__any_sync(0xffffffffu, sees != 0xFFFFu)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = (sees >> i) & 1u ? z[i] : 0xFF800000u;  // -inf
        }
      }
      float mx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mx[i] = fmaxf(fmaxf(__uint_as_float(z[4 * i]), __uint_as_float(z[4 * i + 1])),
                      fmaxf(__uint_as_float(z[4 * i + 2]), __uint_as_float(z[4 * i + 3])));
      float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
      if (half == 0) red_m[buf][th][m] = mt;
      // The weights, against the running maximum as it stands: most tiles leave
      // it, so the exchange with the other warp of the pair ends behind them.
      uint32_t packed[8];
      float alpha = 1.f, lsum, wsum;
      auto weights = [&] {
        const float ref = m_run == -INFINITY ? 0.f : m_run - kLift;
        lsum = wsum = 0.f;  // lsum: times 2^-E, the bits of which are those of 2^E mirrored
        if (!own) {
          const uint64_t nref = pack2(-ref, -ref);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint64_t ls = 0;  // (0, 0)
#pragma unroll
            for (int i = 8 * g; i < 8 * g + 8; i += 2) {
              const float2 d = unpack2(add2(pack2(z[i], z[i + 1]), nref));
              const float2 e = make_float2(ex2(d.x), ex2(d.y));
              packed[i / 2] = h2_bits(__floats2half2_rn(e.x, e.y));
              ls = add2(ls, pack2(e.x, e.y));
            }
            const float2 l2 = unpack2(ls);
            wsum += l2.x + l2.y;
            lsum = fmaf(l2.x + l2.y, __uint_as_float(0x7F000000u - oc[2 * g]), lsum);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            uint32_t f[4], e[4];
            factors(i, f, e);
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = ex2(__uint_as_float(z[i + k]) - ref);
              wsum += x[k];
              lsum = fmaf(x[k], __uint_as_float(0x7F000000u - f[k]), lsum);
            }
            packed[i / 2] = h2_bits(__floats2half2_rn(x[0], x[1]));
            packed[i / 2 + 1] = h2_bits(__floats2half2_rn(x[2], x[3]));
          }
        }
      };
      weights();
      pair_sync(qd);
      mt = fmaxf(mt, red_m[buf][th ^ 1][m]);
      const bool raise = mt > m_run + kLazy || (m_run == -INFINITY && mt > m_run);
      if (__any_sync(0xffffffffu, raise)) {  // (the same in both warps of the pair)
        if (raise) {
          if (m_run != -INFINITY) alpha = ex2(m_run - mt);
          m_run = mt;
        }
        if (__any_sync(0xffffffffu, alpha != 1.f)) {  // (never at a segment's first tile)
          // O is scaled in place.  The stores also rewrite the other lanes
          // (queries, logits) with what they hold, so the products in flight
          // are waited for: PV(t-1), and QK(t+1) if the segment goes on.
          ok = warp_wait(ok, &bar_pv[(t - 1) & 1], ((t - 1) >> 1) & 1, abort);
          if (t + 1 < seg_end)
            ok = warp_wait(ok, &bar_qk[(t + 1) & 1], ((t + 1) >> 1) & 1, abort);
          tc_fence_after();
#pragma unroll 1
          for (int c = 256 * th; c < 256 * th + 256; c += 32) {
            uint32_t v[32];
            tmem_ld_x32_async(tm_q + c, v);
            tmem_ld_wait_regs<32>(v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = half ? __float_as_uint(__uint_as_float(v[i]) * alpha) : v[i];
            tmem_st_x32(tm_q + c, v);
          }
        }
        weights();
      }
      lsum += __shfl_xor_sync(0xffffffffu, lsum, 16);
      l_run = fmaf(l_run, alpha, lsum);  // this warp's half of the tokens
      w_run = fmaf(w_run, alpha, wsum);  // (and this lane's: joined at the end)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int piece = 4 * th + 2 * half + c;
        sts128(p_u + buf * kPBytes + m * 128 + ((piece ^ (m & 7)) << 4), packed[4 * c],
               packed[4 * c + 1], packed[4 * c + 2], packed[4 * c + 3]);
      }
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_p[buf]);
      const uint32_t pv_parity = (t >> 1) & 1;
      ++t;
      if (t < seg_end) continue;

      // ---- the segment's output (in lanes 16-31; a warp has 256 dims) --------
      w_run += __shfl_xor_sync(0xffffffffu, w_run, 16);
      if (half == 0) red_l[th][m] = make_float2(l_run, w_run);
      pair_sync(qd);
      l_run += red_l[th ^ 1][m].x;
      w_run += red_l[th ^ 1][m].y;
      // The next segment's queries first.  (Both warps of the quarter are behind
      // their last scaling of O, which rewrites the queries' lanes too.)
      if (t < ntiles) hs = take_queries();
      ok = warp_wait(ok, &bar_pv[buf], pv_parity, abort);
      tc_fence_after();
      const float ref_out = m_run == -INFINITY ? -INFINITY : m_run - kLift;
      const bool head = t_org >= 0, whole = head && t_org + tiles <= ntiles;
      // A whole unit: out = O / l in bf16.  A part: O / (sum of its weights), at
      // most 6 in magnitude, times 2^13 in fp16: 11 bits down to 2^-27 (an eighth
      // of the output's own rounding; fp32 parts took twice the traffic).  A row's
      // smallest groups lie 2^15 below its largest, and up to 2^19 below the
      // exponent it is held with, and a mean over tokens is smaller again: without
      // the factor they ended in fp16's subnormals (means of 2^-20 were off by up
      // to 3.5 % in rows that CTAs share).
      const float norm = whole ? l_run : w_run;
      const float inv = norm != 0.f ? (whole ? 1.f : kPartScale) / norm : 0.f;
      const int part_slot = 2 * blockIdx.x + (head ? 1 : 0);
      const int64_t dst_row = whole ? out_row : static_cast<int64_t>(part_slot) * kM + m;
      uint16_t* const dst =
          whole ? reinterpret_cast<uint16_t*>(p.out) : reinterpret_cast<uint16_t*>(p.part_o);
#pragma unroll 1
      for (int c0 = 0; c0 < 256; c0 += 64) {
        uint32_t raw[64];
        __syncwarp();
        tmem_ld_x32_async(tm_q + 256 * th + c0, raw);
        tmem_ld_x32_async(tm_q + 256 * th + c0 + 32, raw + 32);
        tmem_ld_wait_regs<64>(raw);
        const float* v = reinterpret_cast<const float*>(raw);
        // 16 rows of 64 dims through 2 KiB of the P buffers (the segment's last PV
        // is done, the next tile's P waits for every worker), so that eight
        // lanes store a row's 128 bytes.
        const uint32_t stage = p_u + warp * 2048;
        if (half == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = v[8 * i + 2 * k] * inv, b = v[8 * i + 2 * k + 1] * inv;
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
              o[k] = whole ? *reinterpret_cast<const uint32_t*>(&h2)
                           : h2_bits(__floats2half2_rn(a, b));
            }
            sts128(stage + (lane & 15) * 128 + ((i ^ (lane & 7)) << 4), o[0], o[1], o[2], o[3]);
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * i + (lane >> 3);
          const int64_t row = __shfl_sync(0xffffffffu, dst_row, r);
          uint32_t o[4];
          lds128(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4), o);
          if (row >= 0)
            *reinterpret_cast<uint4*>(dst + row * kLatent + 256 * th + c0 + 8 * (lane & 7)) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      if (half == 0 && th == 0) {
        if (!whole)
          p.part_ml[part_slot * kM + m] = make_float4(ref_out, l_run, w_run / kPartScale, 0.f);
        else if (p.lse && out_row >= 0)
          p.lse[out_row] = l_run != 0.f ? (ref_out + log2f(l_run)) * 0.69314718055994530942f
                                        : -INFINITY;
      }
      tc_fence_before();  // O is read before the next segment's first PV
      if (t < ntiles) {
        workers_sync();  // (the staging areas are others' P)
        ++u;
        t_org = t;
        enter_segment();
      }
    }
  }
  if (!ok && lane == 0) atomicExch(&g_device_error, kErrWaitTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins the parts of the units that several CTAs shared.  Block (c, y) takes the
// unit whose first part CTA c left and an equal share of its pieces of 8 dims;
// a thread a piece, in one pass over the parts with a running R (a part's loads
// then wait for nothing but the unit's record).
constexpr int kJoinThreads = 256;
// Shares of a unit: many with few units (many loads in flight), fewer with many
// (fewer blocks that find nothing to do).  Measured, whole call, 16 / 8 / 4 shares,
// in us: 1 row of 64 heads over 8,192 tokens 27.7 / 37.2 / 57.0, 31 such rows 84.0 /
// 82.0 / 85.5, 48 114.5 / 114.2 / 113.7; 16 heads over 2,051 tokens, 31 rows 33.6 /
// 34.8 / 39.3, 32 36.1 / 36.3 / 40.0, 64 51.1 / 49.7 / 51.7, 256 144.9 / 142.3 / 143.2.
constexpr int kJoinFew = 32;  // units
constexpr int join_shares(int units) { return units < kJoinFew ? 16 : 8; }
template <bool kSparse>
__global__ void __launch_bounds__(kJoinThreads) k_attn_fp4_combine(const KParams p) {
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x, tid = threadIdx.x;
  const int2 cb = p.comb[c];
  const int parts = cb.y;
  if (parts == 0) return;
  const UnitRows ur = unit_rows<kSparse>(p, cb.x);
  const int hpr = min(p.heads, kM);
  const int pairs = kM / static_cast<int>(gridDim.y);
#pragma unroll 1
  for (int k = tid >> 6; k < pairs; k += kJoinThreads / 64) {
    const int m = static_cast<int>(blockIdx.y) * pairs + k, d = 8 * (tid & 63);
    const int rr = pair_row(m, hpr), h = ur.hg * kM + m - rr * hpr;
    if (rr >= ur.nrows || h >= p.heads) continue;
    const int64_t row = static_cast<int64_t>(ur.row0 + rr) * p.heads + h;
    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float R = -INFINITY, l = 0.f;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      // slot of part i: CTA c's second, then the first of the CTAs behind it
      const int slot = (2 * (c + i) + (i == 0 ? 1 : 0)) * kM + m;
      const uint4 x = *reinterpret_cast<const uint4*>(p.part_o + static_cast<int64_t>(slot) * kLatent + d);
      const float4 ml = p.part_ml[slot];
      const float top = fmaxf(R, ml.x);
      // (a part that saw nothing has R = -inf and zeros, or NaN)
      const float old = R == -INFINITY ? 1.f : ex2(R - top);
      const float w = ml.x == -INFINITY ? 1.f : ex2(ml.x - top);
      R = top;
      l = fmaf(w, ml.y, l * old);
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&in[e]));
        a[2 * e] = fmaf(w * ml.z, f.x, a[2 * e] * old);
        a[2 * e + 1] = fmaf(w * ml.z, f.y, a[2 * e + 1] * old);
      }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(a[2 * e] * inv, a[2 * e + 1] * inv);
      o[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p.out + row * kLatent + d) = make_uint4(o[0], o[1], o[2], o[3]);
    if (d == 0 && p.lse)
      p.lse[row] = l != 0.f ? (R + log2f(l)) * 0.69314718055994530942f : -INFINITY;
  }
}

template <bool kSparse>
bool set_attrs() {
  static std::atomic<bool> attr_set[64];  // zero-initialised: false
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64 && attr_set[dev]) return true;
  if (cudaFuncSetAttribute(k_attn_fp4<kSparse>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemBytes) != cudaSuccess)
    return false;
  if (dev >= 0 && dev < 64) attr_set[dev] = true;
  return true;
}

template <bool kSparse>
cudaError_t launch(const AttnFp4Plan& pl, const KParams& p, cudaStream_t stream) {
  if (!set_attrs<kSparse>()) return cudaGetLastError();
  cudaError_t e = launch_ex(k_attn_fp4<kSparse>, dim3(pl.grid), dim3(kThreads), kSmemBytes, stream,
                            true, 1, p);
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (pl.ws_bytes > 0) {
    e = launch_ex(k_attn_fp4_combine<kSparse>, dim3(pl.grid, join_shares(pl.units)),
                  dim3(kJoinThreads), 0, stream,
                  true, 1, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaGetLastError();
}

constexpr size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

AttnFp4Plan plan_attn_fp4(int rows, int per_seq, int heads, bool sparse, int64_t max_len,
                          int num_sms) {
  AttnFp4Plan pl{};
  pl.groups = (heads + kM - 1) / kM;
  pl.rows_per_unit = sparse || heads > kM / 2 ? 1 : kM / heads;
  if (pl.rows_per_unit > per_seq) pl.rows_per_unit = per_seq;
  pl.rgs = (per_seq + pl.rows_per_unit - 1) / pl.rows_per_unit;
  pl.units = rows / per_seq * pl.rgs * pl.groups;  // (at most 2 x 65535)
  int64_t list = max_len < kFp4MaxTok ? max_len : kFp4MaxTok;  // tokens in a list, at most
  if (sparse && list > kTopK * kPool + kPool - 1) list = kTopK * kPool + kPool - 1;
  int64_t tiles = (list + kTT - 1) / kTT;
  if (tiles < 1) tiles = 1;
  const int sms = num_sms < kMaxGrid ? num_sms : kMaxGrid;
  pl.tiles = pl.units * tiles;  // (below 2^43)
  pl.grid = static_cast<int>(pl.tiles < sms ? pl.tiles : sms);
  if (tiles > 1)  // units of one tile are never split
    pl.ws_bytes = up256(pl.grid * sizeof(int2)) +
                  static_cast<size_t>(2) * pl.grid * (kM * sizeof(float4) + kPartHalfs * 2);
  return pl;
}

cudaError_t launch_attn_fp4(const AttnFp4Plan& pl, const AttnFp4Args& a, cudaStream_t stream) {
  KParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.codes = a.codes;
  p.scales = a.scales;
  p.seq_tok = a.seq_tok;
  p.len_cap = a.len_cap;
  p.idx = a.idx;
  p.count = a.count;
  p.n_vis = a.n_vis;
  p.heads = a.heads;
  p.per_seq = a.per_seq;
  p.units = pl.units;
  p.groups = pl.groups;
  p.rows_per_unit = pl.rows_per_unit;
  p.rgs = pl.rgs;
  p.scale_log2 = a.sm_scale * 1.44269504088896340736f;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  if (pl.ws_bytes > 0) {
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    p.comb = reinterpret_cast<int2*>(ws);
    ws += up256(pl.grid * sizeof(int2));
    p.part_ml = reinterpret_cast<float4*>(ws);
    ws += static_cast<size_t>(2) * pl.grid * kM * sizeof(float4);
    p.part_o = reinterpret_cast<__half*>(ws);
  }
  return a.idx ? launch<true>(pl, p, stream) : launch<false>(pl, p, stream);
}

}  // namespace spx
