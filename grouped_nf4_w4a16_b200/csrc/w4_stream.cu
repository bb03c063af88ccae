// w4_stream.cu -- 4-bit weights times a few activation rows: the kernel behind
// gnf4_gemv (one dense matrix) and gnf4_moe_experts (the experts of a few
// tokens, two launches: gate_up with SwiGLU, then down with the weighted sum).
//
// Passage: package page "grouped-nf4-gemm", "Use this when" (the tail of small
// launches of a decode step, each to be folded away); the page's int4 matrix-
// vector product with 32-wide scales stands beside the grouped GEMM as
// gnf4_gemv's INT4 format.
//
// Mathematics, for a matrix W of N rows with one scale per group of G codes:
//     y[m][n] = sum over groups b of s[n][b] * sum_{k in b} x[m][k] * v[n][k]
// v is the code's value (NF4 table, e2m1, or int4 code minus zero point). The
// inner sum runs on tensor cores (mma.sync m16n8k16, weights as the 16-row
// operand, up to 8 activation rows as the 8 columns, fp32 accumulation); the
// outer sum is one fp32 multiply-add per group.
//   v enters as fp16: exact for e2m1 and int4; NF4 times 1.677654, the scale
//   that keeps the fp16 rounding of all 16 values within 6.0e-5 of the range.
//   x enters as fp16 times a power of two per row that puts the row's largest
//   magnitude in [2^14, 2^15): exact for bf16 elements above 2^-28 of it. The
//   activations between the two launches of gnf4_moe_experts stay fp32 in
//   memory and are rounded to fp16 (2^-11 relative) on the same scale.
//   What the roundings cost: against fp64 the experts' results are off by 1.62e-3
//   to 1.69e-3 in relative norm, the exact ones rounded once to bf16 by 1 % less,
//   the library's five launches (h and every slot's row in bf16) by 2.8e-3 to
//   2.9e-3; a vector product's are off by its bf16 rounding to within 1e-6. One
//   bf16 in ten (NF4 vector product: one in 25) falls to the other side of a
//   rounding border than with fp32 throughout. So NF4 has one part for every
//   row: the decode GEMM's second part for the up rows is half again as many
//   table reads, in a kernel that is bound by them.
//
// Work split. Every warp streams its own share of W and meets the others only
// where a share ends:
//   tile  = 16 weight rows (with SwiGLU 8 gate rows and their 8 up rows).
//   CTA   = a contiguous range of the (batch, tile) pairs; a batch is up to
//           8 NT activation rows of one expert. One CTA per SM.
//   warp  = an equal share of the CTA's tiles x units, laid end to end, cut at
//           any unit (64 or 128 codes). Shares that end inside a tile leave
//           their sums in shared memory, added in share order (deterministic).
//   Each warp feeds a ring of its own (stages of 16 rows x 256 codes, 2 KB, two
//   TMA boxes): no warp waits for another in the stream. (One copy warp with a
//   lane per ring reached 3.9 TB/s, every warp on its own 6.9: a warp's lanes
//   start their copies one after the other.) Batches of more than one column tile of the MMA (NT = 2) read
//   the weights once for 16 rows.
//   The activation rows lie in shared memory for the whole K, or a chunk of it
//   when they do not fit: the CTA then adds its chunks up in fp32, or (vector
//   product, down) the chunks go to different CTAs.
//
// What bounds it (one B200, 6.55 TB/s copy bandwidth; figures of graph replays):
//   MXFP4: issue slots. 85 warp instructions per 1024 codes, 67 % of the issue
//     slots taken; an e2m1 conversion (two codes) runs once a clock and SM, 16
//     of some 32 clocks. 64 tokens x 4 of 128 experts, 2880 x 2880: 345 us for
//     1.47 GB, 4.3 TB/s; 4.7 in the stream itself. (In runs of more than some
//     50 ms the 1 kW power cap takes the SM clock from 1965 to 1820 MHz: 370 us.)
//   NF4: shared memory. Per 1024 codes 16 wavefronts read the value table, 4
//     the codes, 4 the copies write, and the activations; 73 % of the pipe's
//     rate over the whole launch. 5 tokens x 2 of 8 experts, 6144 x 16384: 256
//     us for the 1.0 to 1.2 GB of 6 or 7 experts, over 4 TB/s (275 in long runs).
//   16 rows, NF4, 32768 x 6144: 54.6 us for 114 MB: shared memory again (16 more
//     wavefronts for the rows), and the rows are staged in two chunks of K.
//   Small launches: latency. Of the 24 us of one token x 8 of 64 experts, NF4,
//     2048 x 1024 (28 MB), each launch streams for 3 to 4; tables, staging and
//     the end of the stream take 2 us each, most of it first passes through
//     the code.
//   INT4: the subtraction of zero points and the mantissa trick, 53 % of the
//     ALU pipe; one row, 6144 x 16384, 22.1 us for 53 MB: 384 tiles on 148 SMs,
//     so that a CTA has 2 tiles or 3.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "launch.h"
#include "lut_mma.cuh"

namespace gnf4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
// Stages per warp's ring: 32 KB per SM in flight while one stage a warp is
// read. A third bought nothing (8 rows NF4 32768 x 6144 36.8 us, with three
// 40.7; 5 tokens NF4 258 and 261; 64 tokens MXFP4 349 and 347): the room goes
// to the activation rows, 8 of 6144 at once.
constexpr int kRing = 2;
constexpr int kStageK = 256;          // codes per row and stage
constexpr int kBoxBytes = 1024;       // 8 rows x 128 bytes: one row set of a stage
constexpr int kStageBytes = 2 * kBoxBytes;
constexpr int kLutBytes = 256 * 128;  // fp16 pair per byte, one copy per lane
constexpr int kMaxSlots = GNF4_EXPERTS_MAX_SLOTS;
constexpr int kMaxSplit = 8;          // chunks that CTAs share out
constexpr int kSplitColumns = 32768;  // weight rows up to which they may
constexpr int kMaxRows = 128;         // activation rows staged at once, at most
constexpr int kSmemMax = 227 * 1024;
constexpr float kNf4Scale = 1.6776540f;   // see decode_gemm.cu: the smallest fp16 rounding error
constexpr float kNf4Inv = 1.0f / kNf4Scale;
// The rows are staged 2^14 times too large (their magnitudes end at 2^15);
// the weights' scales carry 2^-14 so that no sum leaves fp32 before the
// result does.
constexpr int kRowShift = 14;
constexpr float kScaleFactor = 1.0f / (1 << kRowShift);

// kSplit, kDownSplit: CTAs work on one chunk of K each
enum Mode : int { kGemv = 0, kSplit = 1, kGateUp = 2, kDown = 3, kDownSplit = 4 };
constexpr bool dense(int mode) { return mode == kGemv || mode == kSplit; }
constexpr bool down(int mode) { return mode == kDown || mode == kDownSplit; }
constexpr bool shared_out(int mode) { return mode == kSplit || mode == kDownSplit; }
enum Fmt : int { kNf4 = 0, kMx = 1, kInt4 = 2 };

struct StreamParams {
  const char *scales;
  const uint8_t *zeros;       // int4 zero points (nullptr: 8)
  int32_t N, K;               // weight rows and codes per row of one matrix
  int32_t MT;                 // tiles per batch
  int32_t chunk, nchunk;      // codes of K staged at once (a multiple of 256), chunks
  int32_t cap;                // rows a batch has at most
  int32_t xrows;              // activation rows the staging area holds (at least cap)
  // copies: row coordinates per tile and per expert, and from the first box to the second
  int32_t tile_rows, expert_rows, box_dx, box_dy;
  // the weight row of box row r of tile t: row_t * t + row_r * r, + row_b in the second box
  int32_t row_t, row_r, row_b;
  const char *x;              // rows of the activations: bf16 (gemv, gate_up) or fp32 (down)
  int64_t x_pitch;            // bytes
  int32_t xvec;               // rows are 16-byte aligned
  const int32_t *ids;         // experts: [T][top_k]
  const float *weights;
  int32_t T, top_k, E, S;     // S = T * top_k (gemv: rows)
  uint16_t *y;                // bf16 result (gemv: [M][ldy], down: [T][N])
  int64_t ldy;
  const uint16_t *bias;       // gemv: bf16 [N] or nullptr
  float *hout;                // gate_up: fp32 [S][N / 2]
  float *part;                // fp32 [rows][N]: sums of the chunks so far; down: every slot's row;
                              // shared out: [chunk][rows][N], the chunks' sums
  uint32_t *counters;         // down: [MT][1 << log_groups] slots done per tile and group of tokens;
                              // kSplit: chunks done per tile of all batches
  int32_t groups, log_groups; // token i is in group i % groups, T or 2^log_groups of them (the lesser)
  float alpha, limit;         // gate_up, clamped form
  int32_t clamped;
  WsHeader *hdr;
};

// ---------------------------------------------------------------- formats
template <int G>
struct Layout {
  static constexpr int kUnitK = G == 128 ? 128 : 64;   // codes per unit
  static constexpr int kUnits = kStageK / kUnitK;      // units per stage
  static constexpr int kUnitGroups = kUnitK / G;       // groups per unit
};

// Scales are fetched a block (1024 codes of a tile's 16 rows) at a time: lane
// l of 32 takes unit l % kUnits of the rows l / kUnits, + kRows, ..., so that
// neighbouring lanes read neighbouring bytes (a lane fetching only what it
// multiplies with touches a line per row and stage, and its loads took issue
// slots from the stream). They wait a block in registers and are then laid out
// in shared memory as the multiply-adds take them, kWords a unit: the scale of
// each group (int4: and its zero point).
template <int FMT, int G, int SF>
struct Scales {
  static constexpr int kBytes = SF == GNF4_SCALE_F32 ? 4 : SF == GNF4_SCALE_BF16 ? 2 : 1;
  static constexpr int kUnits = 1024 / Layout<G>::kUnitK;         // units per block
  static constexpr int kRows = 32 / kUnits;                       // rows per load
  static constexpr int kLoads = 16 / kRows;
  static constexpr int kRaw = kBytes * Layout<G>::kUnitGroups == 8 ? 2 : 1;   // 32-bit words fetched per unit
  static constexpr int kWords = Layout<G>::kUnitGroups * (FMT == kInt4 ? 2 : 1);
  static constexpr int kStageWords = kWords * Layout<G>::kUnits;  // a row's, a multiple of 4
  static constexpr int kPitch = kUnits * kWords + 4;              // words: 8 rows in different banks
  static constexpr int kWarpBytes = 16 * kPitch * 4;
  static __device__ __forceinline__ void fetch(const char *p, uint32_t (&raw)[kRaw]) {
    constexpr int kEntry = kBytes * Layout<G>::kUnitGroups;
    if (kEntry == 2) {
      asm volatile("{\n\t.reg .u16 h;\n\tld.global.nc.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
                   : "=r"(raw[0]) : "l"(p));
    } else {
#pragma unroll
      for (int i = 0; i < kRaw; ++i)
        asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(raw[i]) : "l"(p + 4 * i));
    }
  }
  // Group i of the unit, times kScaleFactor.
  static __device__ __forceinline__ float value(const uint32_t (&raw)[kRaw], int i) {
    if (SF == GNF4_SCALE_E8M0) {   // 2^(s - 127), 255 = NaN
      const uint32_t s = (raw[0] >> (8 * i)) & 255u;
      const float v = s == 255u ? __uint_as_float(0x7FC00000u)
                      : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
      return v * kScaleFactor;
    }
    const uint32_t u = SF == GNF4_SCALE_F32 ? raw[kRaw > 1 ? i : 0]
                                            : (i == 0 ? raw[0] << 16 : raw[0] & 0xFFFF0000u);
    return __uint_as_float(u) * kScaleFactor;
  }
};

// Row of its 8-row box that MMA rows g and g + 8 hold: chosen so that the
// shared-memory reads below hit 32 different banks under the 128-byte swizzle.
template <int G>
__device__ __forceinline__ int box_row(int g) {
  return G == 64 ? ((g & 3) << 1) | (g >> 2) : G == 128 ? ((g & 1) << 2) | (g >> 1) : g;
}

__device__ __forceinline__ uint2 lds_u2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// 16 bytes at a + AT; with SOME only where `on`: elsewhere nothing is read and
// x keeps old values.
template <int AT, bool SOME>
__device__ __forceinline__ void lds_row(uint32_t a, int on, uint32_t (&x)[4]) {
  if (!SOME) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4+%5];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(a), "n"(AT));
    return;
  }
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
               "@p ld.shared.v4.b32 {%0, %1, %2, %3}, [%4+%6];\n\t}"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3])
               : "r"(a), "r"(on), "n"(AT));
}

// byte P of `word` * 128 + base, one instruction
template <int P>
__device__ __forceinline__ uint32_t lut_address(uint32_t word, uint32_t base) {
  uint32_t r;
  asm("dp4a.u32.u32 %0, %1, %2, %3;" : "=r"(r) : "r"(word), "n"(128 << (8 * P)), "r"(base));
  return r;
}

// The 8 codes of `word` as four fp16 pairs. NF4 and e2m1: pair p holds codes
// 2p, 2p + 1; int4: codes p, p + 4 (the activations are staged to match).
template <int FMT>
__device__ __forceinline__ void decode8(uint32_t word, uint32_t lut, uint32_t zero,
                                        uint32_t (&v)[4]) {
  if (FMT == kNf4) {
    asm("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(lut_address<0>(word, lut)));
    asm("ld.shared.b32 %0, [%1];" : "=r"(v[1]) : "r"(lut_address<1>(word, lut)));
    asm("ld.shared.b32 %0, [%1];" : "=r"(v[2]) : "r"(lut_address<2>(word, lut)));
    asm("ld.shared.b32 %0, [%1];" : "=r"(v[3]) : "r"(lut_address<3>(word, lut)));
  } else if (FMT == kMx) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(word));
  } else {
    // code + 1024 as fp16 (the code in the low mantissa bits), minus (zero point + 1024): exact
    const __half2 z = *reinterpret_cast<const __half2 *>(&zero);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t t = ((word >> (4 * p)) & 0x000F000Fu) | 0x64006400u;
      const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&t), z);
      v[p] = *reinterpret_cast<const uint32_t *>(&d);
    }
  }
}

// ------------------------------------------------------------ shared layout
struct Tables {
  uint16_t order[kMaxSlots];       // slots, expert by expert
  uint16_t expert[kMaxSlots];      // per batch
  uint16_t first[kMaxSlots];       // per batch: its first entry of `order`
  uint8_t rows[kMaxSlots];         // per batch
  uint16_t slot_expert[kMaxSlots]; // expert of each slot, 0xFFFF: left out
  uint32_t owed[GNF4_EXPERTS_MAX_TOKENS];   // down: slots per group of tokens (times chunks)
};

struct Shared {
  uint64_t full[kWarps * kRing];   // a stage's copies have landed
  uint64_t never;                  // nothing arrives here (the wait-limit test hook)
  int32_t scan[2 * kWarps];
  int32_t nbatch;
  int32_t abort;
  int32_t sums;                    // down: entries of the list of sums
  uint32_t rowmax[2][kWarps];      // (only rows that several warps stage)
  float rowinv[kMaxRows];
  int32_t rowslot[kMaxRows];
};

constexpr int align_up(int v, int a) { return (v + a - 1) / a * a; }

template <int FMT, int G, int SF, int NT, int MODE>
struct Offsets {
  static constexpr int kScaleOff = kWarps * kRing * kStageBytes;   // (the ring lies at 0)
  static constexpr int kLutOff = kScaleOff + kWarps * Scales<FMT, G, SF>::kWarpBytes;
  static constexpr int kSharedOff = kLutOff + (FMT == kNf4 ? kLutBytes : 0);
  static constexpr int kTablesOff = align_up(kSharedOff + static_cast<int>(sizeof(Shared)), 16);
  static constexpr int kXOff =
      align_up(kTablesOff + (dense(MODE) ? 0 : static_cast<int>(sizeof(Tables))), 128);
};

// ------------------------------------------------------------------ waits
// (32-bit shared addresses)
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0u;
}

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait of a whole warp after a first try failed; the same answer for all lanes.
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, Shared &sh, WsHeader *hdr) {
  const uint32_t hook = hdr->reserved[0];
  const bool ok = wait_bar_lim(bar, parity, reinterpret_cast<volatile int *>(&sh.abort), hdr,
                               hook ? static_cast<uint64_t>(hook) : kTimeoutNs);
  return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------- work split
// Warp w's share of a segment's units (tile by tile) starts at unit
// share_lo(units, w); share_of(units, u) is the share that holds unit u.
// (16 x units < 2^32: a matrix has fewer than 2^23 tiles of at most 2^10
// units, split over the SMs)
__device__ __forceinline__ uint32_t share_lo(uint32_t units, uint32_t w) { return units * w / kWarps; }
__device__ __forceinline__ uint32_t share_of(uint32_t units, uint32_t u) {
  return ((u + 1) * kWarps - 1) / units;
}

// The batches: an expert's rows, `cap` at a time (from the tables), or the
// rows of one matrix, `cap` at a time.
template <int MODE>
struct Batches {
  const Tables &tb;
  int cap, S;
  __device__ __forceinline__ int expert(int b) const { return dense(MODE) ? 0 : tb.expert[b]; }
  __device__ __forceinline__ int first(int b) const { return dense(MODE) ? cap * b : tb.first[b]; }
  __device__ __forceinline__ int rows(int b) const {
    return dense(MODE) ? min(cap, S - cap * b) : tb.rows[b];
  }
};

// Slots by expert and the batches of up to `cap` rows, from the choice of
// experts. Every CTA makes the same tables (a slot's rank within its expert is
// its rank in slot order): the CTAs share out the batches among them.
// Up to 32 slots: one warp, in registers, groups by their first slot (one
// token x 8 experts 25.1 us a layer, by the general case 27.6). False
// if a group has more than `cap` slots (a token naming an expert twice).
__device__ __forceinline__ bool few_tables(const StreamParams &a, Tables &tb, Shared &sh, int e) {
  const int lane = threadIdx.x & 31;
  const bool in = e >= 0 && e < a.E;
  if (!in && e != -1 && blockIdx.x == 0) report_error(a.hdr, GNF4_DEVERR_TOPK, 0);
  const uint32_t below = (1u << lane) - 1u;
  const uint32_t same = __match_any_sync(0xffffffffu, in ? e : -1);
  const int n = __popc(same), rank = __popc(same & below);
  const bool leads = in && rank == 0;
  const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
  if (__any_sync(0xffffffffu, in && n > a.cap)) return false;
  int upto = leads ? n : 0;   // slots of the groups up to this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const int first = __shfl_sync(0xffffffffu, upto - n, __ffs(same) - 1);
  tb.slot_expert[lane] = in ? static_cast<uint16_t>(e) : 0xFFFFu;
  if (in) tb.order[first + rank] = static_cast<uint16_t>(lane);
  if (leads) {
    const int b = __popc(leaders & below);
    tb.expert[b] = static_cast<uint16_t>(e);
    tb.first[b] = static_cast<uint16_t>(first);
    tb.rows[b] = static_cast<uint8_t>(n);
  }
  if (lane == 0) sh.nbatch = __popc(leaders);
  return true;
}

// Bytes of v0 and v1 added up, those of mask only.
__device__ __forceinline__ int byte_sum(const uint4 &v0, const uint4 &v1, uint32_t below) {
  const uint32_t v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  uint32_t n = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // bits 4 i .. 4 i + 3 of `below`, one per byte
    const uint32_t ones = (((below >> (4 * i)) & 15u) * 0x00204081u) & 0x01010101u;
    n = __dp4a(v[i], ones, n);
  }
  return static_cast<int>(n);
}

// The general case, by the whole block. count: 32 bytes per expert, then a word
// per expert; byte w counts the expert's slots among slots 32 w .. 32 w + 31.
__device__ __noinline__ void many_tables(const StreamParams &a, Tables &tb, Shared &sh, char *scratch) {
  constexpr int kEach = (kMaxSlots + kThreads - 1) / kThreads;
  static_assert(kEach * kWarps == 32, "a byte per 32 slots");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint4 *count = reinterpret_cast<uint4 *>(scratch);
  int32_t *base = reinterpret_cast<int32_t *>(scratch + a.E * 32);
#pragma unroll 1
  for (int e = tid; e < 2 * a.E; e += kThreads) count[e] = make_uint4(0u, 0u, 0u, 0u);
  int expert[kEach], before[kEach];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int s = tid + i * kThreads;
    const int32_t e = s < a.S ? a.ids[s] : -1;
    expert[i] = e >= 0 && e < a.E ? e : -1;
    bad |= expert[i] != e && e != -1;
    tb.slot_expert[s] = static_cast<uint16_t>(expert[i]);
  }
  if (bad && blockIdx.x == 0) report_error(a.hdr, GNF4_DEVERR_TOPK, 0);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t same = __match_any_sync(0xffffffffu, expert[i]);
    before[i] = __popc(same & ((1u << lane) - 1u));
    if (expert[i] >= 0 && before[i] == 0)
      reinterpret_cast<uint8_t *>(count)[expert[i] * 32 + i * kWarps + warp] = static_cast<uint8_t>(__popc(same));
  }
  __syncthreads();
  // exclusive sums over the experts: slots and batches
  const int per = (a.E + kThreads - 1) / kThreads;
  int slots = 0, batches = 0;
#pragma unroll 1
  for (int e = tid * per; e < min((tid + 1) * per, a.E); ++e) {
    const int n = byte_sum(count[2 * e], count[2 * e + 1], 0xffffffffu);
    base[e] = n;
    slots += n;
    batches += (n + a.cap - 1) / a.cap;
  }
  int vs = slots, vb = batches;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int x0 = __shfl_up_sync(0xffffffffu, vs, o), x1 = __shfl_up_sync(0xffffffffu, vb, o);
    if (lane >= o) {
      vs += x0;
      vb += x1;
    }
  }
  if (lane == 31) {
    sh.scan[warp] = vs;
    sh.scan[kWarps + warp] = vb;
  }
  __syncthreads();
  int s0 = vs - slots, b0 = vb - batches;
#pragma unroll 1
  for (int w = 0; w < warp; ++w) {
    s0 += sh.scan[w];
    b0 += sh.scan[kWarps + w];
  }
  if (tid == kThreads - 1) sh.nbatch = b0 + batches;
#pragma unroll 1
  for (int e = tid * per; e < min((tid + 1) * per, a.E); ++e) {
    const int n = base[e];
#pragma unroll 1
    for (int r = 0; r < n; r += a.cap, ++b0) {
      tb.expert[b0] = static_cast<uint16_t>(e);
      tb.first[b0] = static_cast<uint16_t>(s0 + r);
      tb.rows[b0] = static_cast<uint8_t>(min(a.cap, n - r));
    }
    base[e] = s0;
    s0 += n;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = expert[i];
    if (e >= 0)
      tb.order[base[e] + byte_sum(count[2 * e], count[2 * e + 1], (1u << (i * kWarps + warp)) - 1u) + before[i]] =
          static_cast<uint16_t>(tid + i * kThreads);
  }
  __syncthreads();
}

// --------------------------------------------------------- activation rows
// 8 consecutive activations of a row as fetched: bf16 in one uint4 (x), fp32
// in two (h, which the launch before wrote).
template <bool F32>
struct Piece {
  uint4 u[F32 ? 2 : 1];
  __device__ __forceinline__ void fetch(const char *row, bool vec, int i) {
    if (F32) {
      const uint4 *p = reinterpret_cast<const uint4 *>(row) + 2 * i;
      u[0] = __ldcg(p);
      u[F32 ? 1 : 0] = __ldcg(p + 1);
    } else if (vec) {
      u[0] = *(reinterpret_cast<const uint4 *>(row) + i);
    } else {
      const uint16_t *p = reinterpret_cast<const uint16_t *>(row) + 8 * i;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = static_cast<uint32_t>(p[2 * j]) | (static_cast<uint32_t>(p[2 * j + 1]) << 16);
      u[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // The largest of m and the magnitudes (fmaxf leaves a NaN out).
  __device__ __forceinline__ float largest(float m) const {
    float v[8];
    widen(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
    return m;
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    const uint4 &l = u[0], &h = u[F32 ? 1 : 0];
    const uint32_t w[8] = {l.x, l.y, l.z, l.w, h.x, h.y, h.z, h.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(F32 ? w[2 * i] : w[i] << 16);
      v[2 * i + 1] = __uint_as_float(F32 ? w[2 * i + 1] : w[i] & 0xFFFF0000u);
    }
  }
};

// Stages `nrows` rows (the segment's batches one after the other, from place
// `first` of the slot order), chunk c, as scaled fp16 in the order the MMA
// fragments read them: the 16-byte piece that lane q takes with word i of a
// unit lies at 4 i + q, so that the four lanes of a row read 64 consecutive
// bytes; the row pitch is 64 modulo 128 bytes. A row is one warp's, or several
// warps' when there are fewer rows than warps. Two passes (the largest
// magnitude, the conversion), kKeep pieces a lane under way at once; where a
// lane has no more than these, they stay in registers in between. Ends with a
// block barrier.
template <int FMT, int G, int MODE>
__device__ __forceinline__ void stage_rows(const StreamParams &a, Shared &sh, const Tables &tb,
                                           char *xs, int pitch, int first, int c, int nrows,
                                           int turn) {
  constexpr bool F32 = down(MODE);
  // (the latency of one more load counts in a vector product alone, the first
  // pass through more code in the short launches of a layer: with 4 / 4 / 4 in
  // place of 4 / 2 / 1 a one-token layer took 24.5 us, not 24.0, one of 64
  // tokens 352, not 348; with 2 a 16-row NF4 product 58.8, not 57.6)
  constexpr int kKeep = dense(MODE) ? 4 : MODE == kGateUp ? 2 : 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int k0 = c * a.chunk, n8 = min(a.chunk, a.K - k0) / 8;
  const int parts = nrows < kWarps ? kWarps / nrows : 1, step = parts * 32;
  // Zero; the next turn's is cleared here, also in turns that use neither: what the turn before
  // left there (read before that turn's last barrier) would scale the next turn's rows.
  uint32_t *rowmax = sh.rowmax[turn & 1];
  if (tid < kWarps) sh.rowmax[(turn & 1) ^ 1][tid] = 0u;
  // (with several warps to a row every warp goes round once, for the barrier)
#pragma unroll 1
  for (int task = warp; parts > 1 ? task == warp : task < nrows; task += kWarps) {
    const int r = task / parts;
    const bool idle = r >= nrows;
    const int slot = idle ? 0 : dense(MODE) ? first + r : tb.order[first + r];
    const char *row = a.x + (MODE == kGateUp ? slot / a.top_k : slot) * a.x_pitch +
                      static_cast<int64_t>(k0) * (F32 ? 4 : 2);
    const int i0 = idle ? n8 : (task - r * parts) * 32 + lane;
    Piece<F32> u[kKeep];
    float m = 0.0f, sc = 0.0f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
      for (int i = i0; i < n8; i += kKeep * step) {
        if (pass == 0 || n8 > kKeep * step) {
#pragma unroll
          for (int j = 0; j < kKeep; ++j)
            if (i + j * step < n8) u[j].fetch(row, a.xvec != 0, i + j * step);
        }
        if (pass == 0) {
#pragma unroll
          for (int j = 0; j < kKeep; ++j)
            if (i + j * step < n8) m = u[j].largest(m);
        } else {
#pragma unroll
          for (int j = 0; j < kKeep; ++j) {
            const int at = i + j * step;
            if (at >= n8) break;
            float v[8];
            u[j].widen(v);
            uint32_t p[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const __half2 h = FMT == kInt4 ? __floats2half2_rn(v[w] * sc, v[w + 4] * sc)
                                             : __floats2half2_rn(v[2 * w] * sc, v[2 * w + 1] * sc);
              p[w] = *reinterpret_cast<const uint32_t *>(&h);
            }
            const int to = G == 64    ? (at & ~7) + 4 * (at & 1) + ((at & 7) >> 1)
                           : G == 128 ? (at & ~15) + 4 * (at & 3) + ((at & 15) >> 2)
                                      : at;
            *reinterpret_cast<uint4 *>(xs + r * pitch + to * 16) = make_uint4(p[0], p[1], p[2], p[3]);
          }
        }
      }
      if (pass == 0) {
        uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (parts > 1) {
          if (lane == 0 && !idle) atomicMax(&rowmax[r], bits);
          __syncthreads();
          bits = rowmax[idle ? 0 : r];
        }
        // a power of two that puts the largest magnitude in [2^14, 2^15)
        const int s = min(141 - static_cast<int>(min(bits >> 23, 254u)), 126);
        sc = __uint_as_float(static_cast<uint32_t>(s + 127) << 23);
        if (lane == 0 && !idle) {
          sh.rowslot[r] = slot;
          sh.rowinv[r] = __uint_as_float(static_cast<uint32_t>(127 - s + kRowShift) << 23) *
                         (FMT == kNf4 ? kNf4Inv : 1.0f);
        }
      }
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- results
template <int NT>
struct Sums {
  float v[NT][4];
};

// The finished sums (C-fragment order) of tile t of the batch whose rows are
// the staged rows row0 .. row0 + nrows - 1, chunk c. One copy out of line: the
// stream's code stays small.
template <int G, int NT, int MODE>
__device__ __noinline__ void finish_tile(const StreamParams &a, const Shared &sh, int t, int c,
                                         int row0, int nrows, const Sums<NT> acc) {
  const int lane = threadIdx.x & 31, g = box_row<G>(lane >> 2), q = lane & 3;
  const bool last = !shared_out(MODE) && c + 1 == a.nchunk;
  // weight rows of the two row sets, and their places in `part`
  const int n0 = MODE == kGateUp ? 8 * t + g : 16 * t + g;
  const int n1 = MODE == kGateUp ? a.N / 2 + n0 : n0 + 8;
  const bool in0 = !dense(MODE) || n0 < a.N, in1 = !dense(MODE) || n1 < a.N;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = 8 * nt + 2 * q + i;
      if (m >= nrows) continue;
      const int slot = sh.rowslot[row0 + m];
      const float inv = sh.rowinv[row0 + m];
      float v0 = acc.v[nt][i] * inv, v1 = acc.v[nt][2 + i] * inv;
      float *p = a.part + (shared_out(MODE) ? static_cast<int64_t>(c) * a.S + slot : slot) * a.N;
      if (!shared_out(MODE) && c > 0) {
        if (in0) v0 += __ldcg(p + n0);
        if (in1) v1 += __ldcg(p + n1);
      }
      if (down(MODE) || !last) {
        if (in0) __stcg(p + n0, v0);
        if (in1) __stcg(p + n1, v1);
      } else if (MODE == kGemv) {
        uint16_t *y = a.y + slot * a.ldy;
        if (a.bias) {
          if (in0) v0 += __uint_as_float(static_cast<uint32_t>(__ldg(a.bias + n0)) << 16);
          if (in1) v1 += __uint_as_float(static_cast<uint32_t>(__ldg(a.bias + n1)) << 16);
        }
        if (in0) y[n0] = bf16_bits(v0);
        if (in1) y[n1] = bf16_bits(v1);
      } else {
        // silu(gate) * up, or clamped: gate * sigmoid(alpha * gate) * (up + 1)
        // (comparisons, not fminf/fmaxf: a NaN goes through)
        float al = 1.0f;
        if (a.clamped) {
          al = a.alpha;
          v0 = v0 > a.limit ? a.limit : v0;
          v1 = (v1 > a.limit ? a.limit : v1 < -a.limit ? -a.limit : v1) + 1.0f;
        }
        a.hout[static_cast<int64_t>(slot) * (a.N / 2) + n0] = v0 / (1.0f + expf(-al * v0)) * v1;
      }
    }
  }
}

// Reports the CTA's tiles [lo, hi), all at once: a count per tile and group of
// tokens tells when the last of the group's slots is there. The CTA that sees
// this puts the group's weighted sums (of the tile's columns) on its list. A
// tile's tokens see their last slots in different CTAs: the sums spread over
// the SMs. (A count per tile, and reports while the stream ran, left a tile's
// whole sum to one CTA and its warps waiting for fences: 377 us for a 64-token
// MXFP4 layer, 371 with these counts; now 366.)
template <int NT>
__device__ __forceinline__ void report_tiles(const StreamParams &a, Shared &sh, const Tables &tb,
                                             uint16_t *list, int lo, int hi) {
  __threadfence();
  constexpr int kAtOnce = 4;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < (hi - lo) * 8 * NT; i0 += kAtOnce * kThreads) {
    int at[kAtOnce];
    uint32_t missing[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int i = i0 + j * kThreads, tile = lo + i / (8 * NT), r = i % (8 * NT), b = tile / a.MT;
      missing[j] = 1u;
      if (tile < hi && r < tb.rows[b]) {
        const int grp = (tb.order[tb.first[b] + r] / a.top_k) & ((1 << a.log_groups) - 1);
        at[j] = (tile - b * a.MT) << a.log_groups | grp;
        missing[j] = tb.owed[grp] - 1u - atomicAdd(a.counters + at[j], 1u);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (missing[j] != 0u) continue;
      a.counters[at[j]] = 0u;   // as the next call wants it
      list[atomicAdd(&sh.sums, 1)] = static_cast<uint16_t>(at[j]);
    }
  }
  __threadfence();
}

// The weighted sums of the list: 4 lanes an entry (tile << log_groups | group),
// 4 columns a lane, kAtOnce slots' loads under way together. (The CTAs that end
// last have most of the sums, up to 600 entries of 4 slots: with the slots
// spread over lanes, in more instructions, that took 10 us.)
template <bool CHUNKS>
__device__ __forceinline__ void combine(const StreamParams &a, const Tables &tb,
                                        const uint16_t *list, int entries) {
  constexpr int kAtOnce = 4;
#pragma unroll 1
  for (int i = threadIdx.x >> 2; i < entries; i += kThreads / 4) {
    const int at = list[i], n = 16 * (at >> a.log_groups) + 4 * (threadIdx.x & 3);
#pragma unroll 1
    for (int tok = at & ((1 << a.log_groups) - 1); tok < a.T; tok += a.groups) {
      const int s0 = tok * a.top_k;
      const float *v0 = a.part + static_cast<int64_t>(s0) * a.N + n;
      const int64_t chunk = static_cast<int64_t>(a.S) * a.N;
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
      for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
        float4 v[kAtOnce];
        float w[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          w[j] = 0.0f;
          v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (j0 + j < a.top_k && tb.slot_expert[s0 + j0 + j] != 0xFFFFu) {
            w[j] = __ldg(a.weights + s0 + j0 + j);
            v[j] = __ldcg(reinterpret_cast<const float4 *>(v0 + static_cast<int64_t>(j0 + j) * a.N));
          }
        }
#pragma unroll 1
        for (int c = 1; CHUNKS && c < a.nchunk; ++c) {   // a slot's row is the sum of its chunks'
          float4 more[kAtOnce];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            more[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (j0 + j < a.top_k && tb.slot_expert[s0 + j0 + j] != 0xFFFFu)
              more[j] = __ldcg(reinterpret_cast<const float4 *>(
                  v0 + c * chunk + static_cast<int64_t>(j0 + j) * a.N));
          }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            v[j].x += more[j].x;
            v[j].y += more[j].y;
            v[j].z += more[j].z;
            v[j].w += more[j].w;
          }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          sum.x = fmaf(w[j], v[j].x, sum.x);
          sum.y = fmaf(w[j], v[j].y, sum.y);
          sum.z = fmaf(w[j], v[j].z, sum.z);
          sum.w = fmaf(w[j], v[j].w, sum.w);
        }
      }
      const uint2 y = make_uint2(static_cast<uint32_t>(bf16_bits(sum.x)) | static_cast<uint32_t>(bf16_bits(sum.y)) << 16,
                                 static_cast<uint32_t>(bf16_bits(sum.z)) | static_cast<uint32_t>(bf16_bits(sum.w)) << 16);
      *reinterpret_cast<uint2 *>(a.y + static_cast<int64_t>(tok) * a.N + n) = y;
    }
  }
}

// kSplit: a count per tile tells when the last of its chunks is there. The CTA
// that sees this adds them up, in their order, a thread 4 columns of a row.
__device__ __forceinline__ void join_chunks(const StreamParams &a, Shared &sh, uint16_t *list, int lo,
                                            int hi) {
  __threadfence();
#pragma unroll 1
  for (int tile = lo + threadIdx.x; tile < hi; tile += kThreads) {
    if (atomicAdd(a.counters + tile, 1u) + 1 != static_cast<uint32_t>(a.nchunk)) continue;
    a.counters[tile] = 0u;   // as the next call wants it
    list[atomicAdd(&sh.sums, 1)] = static_cast<uint16_t>(tile - lo);
  }
  __threadfence();
  __syncthreads();
  const int each = a.cap * 4;
  const int64_t chunk = static_cast<int64_t>(a.S) * a.N;
#pragma unroll 1
  for (int i = threadIdx.x; i < sh.sums * each; i += kThreads) {
    const int at = i / each, r = (i - at * each) >> 2, tile = lo + list[at], b = tile / a.MT;
    const int n = 16 * (tile - b * a.MT) + 4 * (i & 3), row = a.cap * b + r, some = a.N - n;
    if (row >= a.S || some <= 0) continue;
    const float *p = a.part + static_cast<int64_t>(row) * a.N + n;
    float4 v[kMaxSplit], sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c) {
      v[c] = sum;
      if (c >= a.nchunk) continue;
      if (a.N % 4 == 0) {
        v[c] = __ldcg(reinterpret_cast<const float4 *>(p + c * chunk));
      } else {
        v[c].x = __ldcg(p + c * chunk);
        if (some > 1) v[c].y = __ldcg(p + c * chunk + 1);
        if (some > 2) v[c].z = __ldcg(p + c * chunk + 2);
        if (some > 3) v[c].w = __ldcg(p + c * chunk + 3);
      }
    }
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c) {
      sum.x += v[c].x;
      sum.y += v[c].y;
      sum.z += v[c].z;
      sum.w += v[c].w;
    }
    const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= some) continue;
      const float bias = a.bias ? __uint_as_float(static_cast<uint32_t>(__ldg(a.bias + n + j)) << 16) : 0.0f;
      a.y[row * a.ldy + n + j] = bf16_bits(out[j] + bias);
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int FMT, int G, int SF, int NT, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    w4_stream_kernel(const __grid_constant__ CUtensorMap wmap,
                     const __grid_constant__ StreamParams a) {
  using L = Layout<G>;
  using O = Offsets<FMT, G, SF, NT, MODE>;
  using Q = Scales<FMT, G, SF>;
  extern __shared__ char smem_raw[];
  char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Shared &sh = *reinterpret_cast<Shared *>(smem + O::kSharedOff);
  Tables &tb = *reinterpret_cast<Tables *>(smem + O::kTablesOff);
  char *xs = smem + O::kXOff;
  const int tid = threadIdx.x, lane = tid & 31;
  // (a reduction's result is known to be the same in a warp: what follows from it is kept once
  // per warp, not per lane)
  const int warp = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(tid) >> 5));

  if (tid <= kWarps * kRing) mbar_init(&sh.full[tid], 1);   // (the last one is `never`)
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (tid < 2 * kWarps) sh.rowmax[0][tid] = 0u;
  if (tid == 0) {
    sh.abort = 0;
    sh.sums = 0;
    sh.nbatch = (a.S + a.cap - 1) / a.cap;   // (of one matrix)
  }
  if (FMT == kNf4) {
    // table row b, copy l: the pair of byte b's values (even k in the high nibble)
#pragma unroll 1
    for (int i = tid; i < 256 * 8; i += kThreads) {
      const int b = i >> 3;
      const uint32_t p = half_bits(nf4_value(b >> 4) * kNf4Scale) |
                         (half_bits(nf4_value(b & 15) * kNf4Scale) << 16);
      reinterpret_cast<uint4 *>(smem + O::kLutOff)[i] = make_uint4(p, p, p, p);
    }
  }

  // Inputs may come from the kernel before. The down launch follows its
  // gate_up launch, which lets it start only after its own wait: what came
  // before both (the choice of experts, the weights) is complete by then, so
  // only what gate_up writes has to be waited for, further below.
  if (!down(MODE)) {
    pdl_wait();
    pdl_trigger();
  }
  if (!dense(MODE)) {
    if (down(MODE) && tid < GNF4_EXPERTS_MAX_TOKENS) tb.owed[tid] = 0u;
    bool few = a.S <= 32;
    if (few) {
      if (warp == 0) {
        const bool ok = few_tables(a, tb, sh, lane < a.S ? a.ids[lane] : -1);
        if (!ok && lane == 0) sh.nbatch = -1;
      }
      __syncthreads();
      few = sh.nbatch >= 0;
    }
    if (!few) many_tables(a, tb, sh, xs);
    if (down(MODE)) {
#pragma unroll 1
      for (int s = tid; s < a.S; s += kThreads)
        if (tb.slot_expert[s] != 0xFFFFu)
          atomicAdd(&tb.owed[(s / a.top_k) & ((1 << a.log_groups) - 1)],
                    MODE == kDownSplit ? static_cast<uint32_t>(a.nchunk) : 1u);
    }
  } else {
    __syncthreads();
  }
  const int nbatch = sh.nbatch;
  const Batches<MODE> bt{tb, a.cap, a.S};
  // The CTA's tiles [lo, hi) of all (batch, tile) pairs, batch by batch.
  // (tiles x CTAs < 2^32: see share_lo)
  const uint32_t total = static_cast<uint32_t>(nbatch) * static_cast<uint32_t>(a.MT);
  int lo, hi, c0 = 0;   // c0: the first chunk
  if (shared_out(MODE)) {
    const uint32_t ctas = gridDim.x / a.nchunk, rank = blockIdx.x % ctas;
    lo = static_cast<int>(total * rank / ctas);
    hi = static_cast<int>(total * (rank + 1) / ctas);
    c0 = static_cast<int>(blockIdx.x / ctas);
  } else {
    lo = static_cast<int>(total * blockIdx.x / gridDim.x);
    hi = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  }

  const int g = lane >> 2, q = lane & 3, br = box_row<G>(g);
  const int pitch = a.chunk * 2 + 64, kg = a.K / G;   // kg: groups per row
  const uint32_t lut = smem_u32(smem + O::kLutOff) + lane * 4;
  const uint32_t xlane = smem_u32(xs) + q * 16;
  const uint32_t ring = smem_u32(smem) + warp * (kRing * kStageBytes);
  const uint32_t full = smem_u32(sh.full + warp * kRing);
  // this lane's words of unit 0 within a stage; unit i: XOR i << 5 (i << 6 with 128-code units)
  const uint32_t wlane =
      br * 128 + (G == 32   ? ((br & 7) << 4) + q * 4
                  : G == 64 ? ((((q >> 1) ^ (br & 7)) << 4) + (q & 1) * 8)
                            : ((q ^ (br & 7)) << 4));
  const uint32_t scales = smem_u32(smem + O::kScaleOff) + warp * Q::kWarpBytes;
  uint32_t slot = 0u, phase = 0u;   // of the stage to multiply next
  int turn = 0;                     // stagings so far
  bool alive = true;
  uint32_t xb[NT][2][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 8; ++i) xb[nt][i / 4][i % 4] = 0u;

  // A segment is a run of tiles whose batches' activation rows fit the staging
  // area together (most often all of the CTA's), for one chunk of K.
#pragma unroll 1
  for (int from = lo, end = lo, c = shared_out(MODE) ? c0 : a.nchunk - 1;;) {
    if (shared_out(MODE) || ++c == a.nchunk) {
      if (!shared_out(MODE)) c = 0;
      from = end;
      if (from >= hi) break;
      int b = from / a.MT, rows = bt.rows(b);
      end = (b + 1) * a.MT;
      while (end < hi && rows + bt.rows(b + 1) <= a.xrows) {
        ++b;
        rows += bt.rows(b);
        end += a.MT;
      }
      end = min(end, hi);
    }
    const int b0 = from / a.MT, b1 = (end - 1) / a.MT;
    const int first0 = bt.first(b0), srows = bt.first(b1) + bt.rows(b1) - first0;
    const int nblk = min(a.chunk, a.K - c * a.chunk) / L::kUnitK;
    const uint32_t units = static_cast<uint32_t>((end - from) * nblk), u0 = share_lo(units, warp);
    int left = static_cast<int>(share_lo(units, warp + 1) - u0);   // units of the share to come
    int kb = static_cast<int>(u0 % nblk);
    const int tile0 = from + static_cast<int>(u0 / nblk);
    int b = tile0 / a.MT, t = tile0 - b * a.MT;
    const bool cut0 = left > 0 && (kb != 0 || left < nblk);   // the first piece is no whole tile
    bool at_first = true, cut1 = false;   // cut1: neither is the last one

    // ---- ahead of the multiplication: copies of the codes, kRing stages
    int a_left = left, a_b = b, a_t = t, a_kb = kb, a_run = 0, a_x = 0, a_row = 0;
    int flying = 0;   // stages asked for and not multiplied
    auto refill = [&](uint32_t dst, uint32_t bar) __attribute__((always_inline)) {
      if (a_run <= 0) {   // to tile a_t of batch a_b, from unit a_kb
        if (a_left == 0) {
          --flying;
          return;
        }
        a_run = min(a_left, nblk - a_kb);
        a_left -= a_run;
        a_x = (c * a.chunk + a_kb * L::kUnitK) / 2;
        a_row = bt.expert(a_b) * a.expert_rows + a_t * a.tile_rows;
        a_kb = 0;
        if (++a_t == a.MT) {
          a_t = 0;
          ++a_b;
        }
      }
      if (elect_one()) {
        expect_bytes(bar, kStageBytes);
        tma_box(dst, &wmap, a_x, a_row, bar);
        tma_box(dst + kBoxBytes, &wmap, a_x + a.box_dx, a_row + a.box_dy, bar);
      }
      a_x += kStageK / 2;
      a_run -= L::kUnits;
    };
    // ---- and the scales of the next block
    uint32_t raw[Q::kLoads][Q::kRaw], rawz[Q::kLoads];
    int s_left = left, s_b = b, s_t = t, s_kb = kb;
    auto fetch_block = [&]() {
      if (s_left == 0) return;
      const int n = min(min(Q::kUnits, s_left), nblk - s_kb);
      const int e = bt.expert(s_b), unit = lane % Q::kUnits, r = lane / Q::kUnits;
      const int n0 = a.row_t * s_t + a.row_r * r;   // weight row of the first load
      const int64_t at = (static_cast<int64_t>(e) * a.N + n0) * kg +
                         (c * a.chunk + (s_kb + unit) * L::kUnitK) / G;
      const int step = a.row_r * Q::kRows;
#pragma unroll
      for (int i = 0; i < Q::kLoads; ++i) {
        const int more = step * (i % (Q::kLoads / 2)) + (i >= Q::kLoads / 2 ? a.row_b : 0);
        if (unit < n && (!dense(MODE) || n0 + more < a.N)) {
          const int64_t j = at + static_cast<int64_t>(more) * kg;
          Q::fetch(a.scales + j * Q::kBytes, raw[i]);
          if (FMT == kInt4) {
            rawz[i] = 0x0808u;
            if (a.zeros)
              rawz[i] = L::kUnitGroups == 2 ? *reinterpret_cast<const uint16_t *>(a.zeros + j) : a.zeros[j];
          }
        }
      }
      s_left -= n;
      s_kb += n;
      if (s_kb == nblk) {
        s_kb = 0;
        if (++s_t == a.MT) {
          s_t = 0;
          ++s_b;
        }
      }
    };
    auto put_block = [&]() {
      const uint32_t to = scales + ((lane / Q::kUnits) * Q::kPitch + (lane % Q::kUnits) * Q::kWords) * 4;
#pragma unroll
      for (int i = 0; i < Q::kLoads; ++i) {
#pragma unroll
        for (int j = 0; j < L::kUnitGroups; ++j) {
          const uint32_t dst = to + (i * Q::kRows * Q::kPitch + j * (Q::kWords / L::kUnitGroups)) * 4;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(Q::value(raw[i], j)) : "memory");
          if (FMT == kInt4) {   // 1024 + zero point twice: fp16 bits 0x6400 + z up to 255
            const uint32_t z = (0x6400u + ((rawz[i] >> (8 * j)) & 255u)) * 0x10001u;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 4), "r"(z) : "memory");
          }
        }
      }
    };

    Sums<NT> acc, held;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc.v[nt][i] = held.v[nt][i] = 0.0f;

    {
      uint32_t sl = slot;
#pragma unroll 1
      for (int i = 0; i < kRing; ++i) {
        ++flying;
        refill(ring + sl * kStageBytes, full + sl * 8);
        sl = sl + 1 == kRing ? 0u : sl + 1;
      }
    }
    fetch_block();

    if (down(MODE) && turn == 0) {
      pdl_wait();
      pdl_trigger();
    }
    __syncthreads();   // the staging area is free
    if (__any_sync(0xffffffffu, sh.abort != 0)) alive = false;
    stage_rows<FMT, G, MODE>(a, sh, tb, xs, pitch, first0, c, srows, turn);
    // Test hook: a non-zero word 2 of the header makes the first wait one that
    // nothing ends, limited to that many nanoseconds.
    if (turn == 0 && *reinterpret_cast<const volatile uint32_t *>(&a.hdr->reserved[0]) != 0u)
      alive = wait_slow(&sh.never, 0u, sh, a.hdr);
    ++turn;

#pragma unroll 1
    while (left > 0 && alive) {
      // ---- one piece: `piece` units of tile t of batch b from unit kb
      int piece = min(left, nblk - kb);
      left -= piece;
      const bool ends = kb + piece == nblk;
      const int row0 = bt.first(b) - first0, nrows = bt.rows(b);
      // lane row g feeds column g of the MMA; the registers of columns past
      // the batch hold old values, and nothing reads their results
      int mine[NT];
      uint32_t xat[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mine[nt] = 8 * nt + g < nrows;
        const int r = NT == 1 || mine[nt] ? 8 * nt + g : 0;   // (some row of the batch)
        xat[nt] = xlane + (row0 + r) * pitch + kb * (L::kUnitK * 2);
      }
      kb = 0;
#pragma unroll 1
      do {
        // ---- one block of scales of it
        int m = min(piece, Q::kUnits);
        piece -= m;
        put_block();
        __syncwarp();
        fetch_block();
        uint32_t sat = scales + br * Q::kPitch * 4;
#pragma unroll 1
        do {
          // ---- one stage
          const int n = min(m, L::kUnits);
          // this lane's scales: rows br and 8 + br
          uint32_t f0[Q::kStageWords], f1[Q::kStageWords];
#pragma unroll
          for (int i = 0; i < Q::kStageWords; i += 4) {
            const uint4 u = lds_u4(sat + i * 4), v = lds_u4(sat + (8 * Q::kPitch + i) * 4);
            f0[i] = u.x; f0[i + 1] = u.y; f0[i + 2] = u.z; f0[i + 3] = u.w;
            f1[i] = v.x; f1[i + 1] = v.y; f1[i + 2] = v.z; f1[i + 3] = v.w;
          }
          const uint32_t bar = full + slot * 8, stage = ring + slot * kStageBytes;
          const bool ok = try_wait(bar, phase);
          if (!__all_sync(0xffffffffu, ok)) {
            alive = wait_slow(sh.full + warp * kRing + slot, phase, sh, a.hdr);
            if (!alive) goto gave_up;
          }
          uint32_t wpart = stage + wlane;
          auto unit = [&](auto ic) __attribute__((always_inline)) {
            constexpr int I = decltype(ic)::value;
            constexpr int i = I;
            constexpr int kWords = L::kUnitK / 32;            // words per lane and row
            constexpr int kPerGroup = G == 32 ? 1 : kWords;   // of which one group holds
            uint32_t wa[kWords], wb[kWords];
            // (XOR on the whole address: the ring starts on 1024 bytes)
            if (G == 32) {
  #pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t at = wpart ^ ((2 * i + j) << 4);
                wa[j] = lds_u32(at);
                wb[j] = lds_u32(at + kBoxBytes);
              }
            } else if (G == 64) {
              const uint32_t at = wpart ^ (i << 5);
              const uint2 va = lds_u2(at), vb = lds_u2(at + kBoxBytes);
              wa[0] = va.x; wa[1] = va.y;
              wb[0] = vb.x; wb[1] = vb.y;
            } else {
              const uint32_t at = wpart ^ (i << 6);
              const uint4 va = lds_u4(at), vb = lds_u4(at + kBoxBytes);
              wa[0] = va.x; wa[1] = va.y; wa[kWords - 2] = va.z; wa[kWords - 1] = va.w;
              wb[0] = vb.x; wb[1] = vb.y; wb[kWords - 2] = vb.z; wb[kWords - 1] = vb.w;
            }
  #pragma unroll
            for (int gr = 0; gr < kWords / kPerGroup; ++gr) {
              // words of the group within the stage's (a dynamic unit only in the rolled loop below)
              const int gi = (i * L::kUnitGroups + gr) * (Q::kWords / L::kUnitGroups);
              const uint32_t zp0 = FMT == kInt4 ? f0[gi + (FMT == kInt4 ? 1 : 0)] : 0u;
              const uint32_t zp1 = FMT == kInt4 ? f1[gi + (FMT == kInt4 ? 1 : 0)] : 0u;
              float d[NT][4];
  #pragma unroll
              for (int j = 0; j < kPerGroup; ++j) {
                const int w = gr * kPerGroup + j;
                uint32_t pa[4], pb[4];
                decode8<FMT>(wa[w], lut, zp0, pa);
                decode8<FMT>(wb[w], lut, zp1, pb);
  #pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  // (up to 8 rows: only the lanes of the batch's rows read, fewer bytes from
                  // shared memory; more: nearly all have one, and loads without a predicate
                  // leave the registers freer: 54.0 us against 55.4 for 16 rows, NF4,
                  // 32768 x 6144, 52.4 against 51.5 for 9; up to 8 rows 291 against 278
                  // for 5 tokens of 6144 x 16384)
                  constexpr int kAt = I * (L::kUnitK * 2);
                  uint32_t (&x)[4] = xb[nt][w % 2];
                  if (w == 0) lds_row<kAt, NT == 1>(xat[nt], mine[nt], x);
                  else if (w == 1) lds_row<kAt + 64, NT == 1>(xat[nt], mine[nt], x);
                  else if (w == 2) lds_row<kAt + 128, NT == 1>(xat[nt], mine[nt], x);
                  else lds_row<kAt + 192, NT == 1>(xat[nt], mine[nt], x);
                  if (j == 0)
                    mma_f16_z(d[nt], pa[0], pb[0], pa[1], pb[1], x[0], x[1]);
                  else
                    mma_f16(d[nt], pa[0], pb[0], pa[1], pb[1], x[0], x[1]);
                  mma_f16(d[nt], pa[2], pb[2], pa[3], pb[3], x[2], x[3]);
                }
              }
              const float sa = __uint_as_float(f0[gi]), sb = __uint_as_float(f1[gi]);
  #pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                acc.v[nt][0] = fmaf(d[nt][0], sa, acc.v[nt][0]);
                acc.v[nt][1] = fmaf(d[nt][1], sa, acc.v[nt][1]);
                acc.v[nt][2] = fmaf(d[nt][2], sb, acc.v[nt][2]);
                acc.v[nt][3] = fmaf(d[nt][3], sb, acc.v[nt][3]);
              }
            }
          };
          // (a whole stage as straight-line code: the units' loads and products overlap)
          if (n == L::kUnits) {
            unit(std::integral_constant<int, 0>{});
            unit(std::integral_constant<int, 1>{});
            if constexpr (L::kUnits > 2) {
              unit(std::integral_constant<int, 2>{});
              unit(std::integral_constant<int, 3>{});
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) xat[nt] += kStageK * 2;
          } else {
            // one unit at a time: its scales and activations move to the front
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
              unit(std::integral_constant<int, 0>{});
              wpart ^= ((i ^ (i + 1)) << (G == 128 ? 6 : 5));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) xat[nt] += L::kUnitK * 2;
#pragma unroll
              for (int j = 0; j + Q::kWords < Q::kStageWords; ++j) {
                f0[j] = f0[j + Q::kWords];
                f1[j] = f1[j + Q::kWords];
              }
            }
          }
          __syncwarp();   // the slot is read: it is refilled
          refill(stage, bar);
          sat += Q::kStageWords * 4;
          m -= L::kUnits;
          if (++slot == kRing) {
            slot = 0u;
            phase ^= 1u;
          }
        } while (m > 0);
      } while (piece > 0);

      if (at_first ? !cut0 : ends) {   // a whole tile
        finish_tile<G, NT, MODE>(a, sh, t, c, row0, nrows, acc);
      } else if (at_first) {
        held = acc;
      } else {
        cut1 = true;   // the share's last piece: stays in acc
        break;
      }
      at_first = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.v[nt][i] = 0.0f;
      if (++t == a.MT) {
        t = 0;
        ++b;
      }
    }
  gave_up:
    // after a wait that gave up: copies still under way land before the CTA ends
    if (!alive && lane == 0) {
      for (; flying > 0; --flying) {
        drain_wait(sh.full + warp * kRing + slot, phase);
        if (++slot == kRing) {
          slot = 0u;
          phase ^= 1u;
        }
      }
    }

    // ---- cut tiles: every share's pieces through shared memory, added in order
    __syncthreads();   // the activation rows are read
    float4 *pieces = reinterpret_cast<float4 *>(xs);   // [warp][first, last][NT][32]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (cut0)
        pieces[((warp * 2) * NT + nt) * 32 + lane] =
            make_float4(held.v[nt][0], held.v[nt][1], held.v[nt][2], held.v[nt][3]);
      if (cut1)
        pieces[((warp * 2 + 1) * NT + nt) * 32 + lane] =
            make_float4(acc.v[nt][0], acc.v[nt][1], acc.v[nt][2], acc.v[nt][3]);
    }
    __syncthreads();
    const bool good = sh.abort == 0;
#pragma unroll 1
    for (int tile = from + warp; tile < end; tile += kWarps) {
      // shares that hold its units [ua, ua + nblk): cut if more than one does
      const uint32_t ua = static_cast<uint32_t>((tile - from) * nblk);
      const uint32_t w0 = share_of(units, ua), w1 = share_of(units, ua + nblk - 1);
      if (w0 == w1 || !good) continue;   // finished by its warp
      Sums<NT> sum;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum.v[nt][i] = 0.0f;
#pragma unroll 1
      for (uint32_t w = w0; w <= w1; ++w) {
        const uint32_t start = share_lo(units, w);
        if (start == share_lo(units, w + 1)) continue;
        const int which = start >= ua ? 0 : 1;   // the share's first piece or its last
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float4 v = pieces[((w * 2 + which) * NT + nt) * 32 + lane];
          sum.v[nt][0] += v.x;
          sum.v[nt][1] += v.y;
          sum.v[nt][2] += v.z;
          sum.v[nt][3] += v.w;
        }
      }
      const int tb_ = tile / a.MT, tt = tile - tb_ * a.MT;
      finish_tile<G, NT, MODE>(a, sh, tt, c, bt.first(tb_) - first0, bt.rows(tb_), sum);
    }
  }

  if (MODE == kSplit) {
    __syncthreads();
    if (sh.abort == 0) join_chunks(a, sh, reinterpret_cast<uint16_t *>(xs), lo, hi);
  }
  if (down(MODE)) {
    if (turn == 0) {   // no tiles here
      pdl_wait();
      pdl_trigger();
    }
    __syncthreads();
    if (sh.abort == 0) {
      uint16_t *list = reinterpret_cast<uint16_t *>(xs);   // (nothing reads the rows any more)
      report_tiles<NT>(a, sh, tb, list, lo, hi);
      __syncthreads();
      combine<MODE == kDownSplit>(a, tb, list, sh.sums);
    }
    // tokens whose slots are all left out
#pragma unroll 1
    for (int grp = blockIdx.x; grp < a.groups; grp += gridDim.x) {
      if (tb.owed[grp] != 0u) continue;
      for (int tok = grp; tok < a.T; tok += a.groups)
        for (int i = tid; i < a.N; i += kThreads) a.y[static_cast<int64_t>(tok) * a.N + i] = 0;
    }
  }
}

// ------------------------------------------------------------------ launch
using Kernel = void (*)(const CUtensorMap, const StreamParams);

struct Variant {
  Kernel kernel;
  int xoff;
  int id;   // below kVariants
};

template <int FMT, int G, int SF, int NT, int MODE>
Variant variant(int id) {
  return {w4_stream_kernel<FMT, G, SF, NT, MODE>, Offsets<FMT, G, SF, NT, MODE>::kXOff, id};
}

template <int FMT, int G, int SF, int MODE>
Variant pick_nt(int nt, int id) {
  return nt == 1 ? variant<FMT, G, SF, 1, MODE>(id) : variant<FMT, G, SF, 2, MODE>(id + 1);
}

template <int FMT, int G, int MODE>
Variant pick_sf(int sf, int nt, int id) {
  return sf == GNF4_SCALE_F32 ? pick_nt<FMT, G, GNF4_SCALE_F32, MODE>(nt, id)
                              : pick_nt<FMT, G, GNF4_SCALE_BF16, MODE>(nt, id + 2);
}

constexpr int kVariants = 45;

template <int MODE>
Variant pick_gemv(int fmt, int group, int sf, int nt, int id) {
  if (fmt == GNF4_FMT_NF4) return pick_sf<kNf4, 64, MODE>(sf, nt, id);
  if (fmt == GNF4_FMT_MXFP4) return pick_nt<kMx, 32, GNF4_SCALE_E8M0, MODE>(nt, id + 4);
  if (group == 32) return pick_sf<kInt4, 32, MODE>(sf, nt, id + 6);
  if (group == 64) return pick_sf<kInt4, 64, MODE>(sf, nt, id + 10);
  return pick_sf<kInt4, 128, MODE>(sf, nt, id + 14);
}

template <int MODE>
Variant pick_experts(int fmt, int sf, int id) {
  if (fmt == GNF4_FMT_MXFP4) return variant<kMx, 32, GNF4_SCALE_E8M0, 1, MODE>(id);
  return sf == GNF4_SCALE_F32 ? variant<kNf4, 64, GNF4_SCALE_F32, 1, MODE>(id + 1)
                              : variant<kNf4, 64, GNF4_SCALE_BF16, 1, MODE>(id + 2);
}

// Codes of K per chunk for `rows` activation rows in `area` bytes.
int32_t chunk_of(int32_t K, int rows, int area) {
  int64_t fit = (static_cast<int64_t>(area) / rows - 64) / 2 / kStageK * kStageK;
  if (fit < kStageK) fit = kStageK;
  if (K <= fit) return (K + kStageK - 1) / kStageK * kStageK;
  const int64_t n = (K + fit - 1) / fit;
  const int64_t each = (K + n - 1) / n;
  return static_cast<int32_t>((each + kStageK - 1) / kStageK * kStageK);
}

// Whether the chunks of K of a vector product go to different CTAs, each
// staging one, their sums joined through memory: when its rows take several
// chunks, or its tiles leave many SMs a tile short. In microseconds: a CTA
// reads a tile's 8 K bytes in K / 3750; a chunk in turn costs 5 (its staging,
// the cut tiles, the ring's start); the join 2.5, and 1 for every 512 pieces of
// 4 columns that a CTA may have to add up.
// Chunks in turn and split, measured for NF4, MXFP4 and INT4 in groups of 128.
// Split by the rule: 16 rows 6144 x 16384 64.1 and 34.9, 65.6 and 30.6, 54.8
// and 31.8; 16 rows 2048 x 8192 30.6 and 16.3, 30.8 and 15.6, 24.0 and 15.7; 8
// rows 4096 x 14336 32.3 and 20.3, 25.6 and 18.7, 27.2 and 19.1; 32 rows 2048 x
// 8192 31.8 and 23.5, 31.8 and 23.0, 25.2 and 18.0. In turn by it: 1 row 6144 x
// 16384 21.9 and 23.6, 19.1 and 20.2, 21.7 and 22.4; 1 row 2048 x 2048 7.0 and
// 8.8, 7.5 and 9.1, 7.0 and 8.5; 32 rows 16384 x 4096 38.2 and 38.9, 37.0 and
// 35.9, 31.0 and 36.3. Its constants are NF4's, and it misses some percent
// where many tiles are joined: 16 rows 32768 x 6144 54.4 and 53.5, 51.0 and
// 48.8, 50.4 and 47.9; 24 rows 86.8 and 85.9, 81.6 and 78.5, 83.4 and 80.0; 8
// rows INT4 8192 x 8192 20.8 and 19.4.
bool choose_split(StreamParams &p, int area) {
  if (p.N > kSplitColumns) return false;
  const int sms = device_sm_count();
  const int64_t tiles = static_cast<int64_t>((p.S + p.cap - 1) / p.cap) * p.MT;
  const auto per_cta = [&](int64_t ctas) { return static_cast<double>((tiles + ctas - 1) / ctas); };
  const int32_t whole = chunk_of(p.K, p.cap, area);
  double best = per_cta(sms) * p.K / 3750 + 5.0 * ((p.K + whole - 1) / whole - 1);
  bool split = false;
  for (int n = 2; n <= kMaxSplit && n <= sms; ++n) {
    const int32_t chunk = ((p.K + n - 1) / n + kStageK - 1) / kStageK * kStageK;
    if ((p.K + chunk - 1) / chunk != n || static_cast<int64_t>(p.cap) * (chunk * 2 + 64) > area) continue;
    const double mine = per_cta(sms / n), with = mine * chunk / 3750 + 2.5 + mine * p.cap * 4 / 512;
    if (with >= best) continue;
    best = with;
    split = true;
    p.chunk = chunk;
    p.nchunk = n;
  }
  return split;
}

cudaError_t launch(const Variant &v, int mode, int nt, const uint8_t *w, int64_t wrows,
                   int64_t row_bytes, StreamParams &p, cudaStream_t stream) {
  CUtensorMap map;
  if (!encode_tensor_map_2d(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w,
                            static_cast<uint64_t>(row_bytes), static_cast<uint64_t>(wrows),
                            static_cast<uint64_t>(row_bytes), 128, 8, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  // Bytes for the activation rows; the sums of cut tiles (two per warp of 16 x
  // 8 NT fp32), while the tables are built 36 bytes per expert, and at the
  // end the list of sums to make, take turns with them.
  const int area = kSmemMax - 1024 - v.xoff;
  if (!shared_out(mode)) {
    p.chunk = chunk_of(p.K, p.cap, area);
    p.nchunk = (p.K + p.chunk - 1) / p.chunk;
  }
  const int sms = device_sm_count(), grid = shared_out(mode) ? sms / p.nchunk * p.nchunk : sms;
  p.xrows = std::min(kMaxRows, area / (p.chunk * 2 + 64));
  const int need = std::max(std::max(std::min(p.xrows, p.S) * (p.chunk * 2 + 64),
                                     kWarps * 2 * nt * 512),
                            std::max(dense(mode) ? 0 : p.E * 36, down(mode) ? (p.MT << p.log_groups) * 2 : 0));
  // (a split's list of tiles, 2 bytes each of at most 4096, takes less than the cut tiles)
  const size_t bytes = static_cast<size_t>(1024 + v.xoff + need);
  static bool configured[64][kVariants] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || !configured[dev][v.id]) {
    err = cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64) configured[dev][v.id] = true;
  }
  return launch_pdl(v.kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), bytes,
                    stream, map, p);
}

}  // namespace

size_t gemv_workspace_bytes(int64_t M, int32_t N) {
  // the sums of the chunks so far, or of every chunk of a split
  const size_t columns = std::max<size_t>(N, static_cast<size_t>(kMaxSplit) * std::min(N, kSplitColumns));
  return kStreamPrefixBytes + (static_cast<size_t>(M) * columns * 4 + 255) / 256 * 256;
}

size_t experts_workspace_bytes(int64_t S, int32_t H, int32_t F) {
  // h; then gate_up's sums of the chunks so far, or the slots' rows of every chunk of F
  const size_t h = (static_cast<size_t>(S) * F * 4 + 255) / 256 * 256;
  const int area = kSmemMax - 1024 - Offsets<kNf4, 64, GNF4_SCALE_F32, 1, kDown>::kXOff;   // (the smallest)
  const size_t chunks = std::min((F - 1) / chunk_of(F, 8, area) + 1, kMaxSplit);
  const size_t columns = std::max<size_t>(2 * static_cast<size_t>(F), chunks * H);
  const size_t part = (static_cast<size_t>(S) * columns * 4 + 255) / 256 * 256;
  return kStreamPrefixBytes + h + part;
}

cudaError_t launch_gemv(const gnf4_gemv_desc &d, void *workspace, cudaStream_t stream) {
  StreamParams p = {};
  p.scales = static_cast<const char *>(d.scales);
  p.zeros = d.zeros;
  p.N = d.N;
  p.K = d.K;
  p.MT = (d.N + 15) / 16;
  p.tile_rows = p.row_t = 16;
  p.row_r = 1;
  p.box_dy = p.row_b = 8;
  p.x = reinterpret_cast<const char *>(d.x);
  p.x_pitch = d.ldx * 2;
  p.xvec = reinterpret_cast<uintptr_t>(d.x) % 16 == 0 && d.ldx % 8 == 0;
  p.S = d.M;
  p.y = d.y;
  p.ldy = d.ldy;
  p.bias = d.bias;
  p.hdr = static_cast<WsHeader *>(workspace);
  p.counters = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + kWsHeaderBytes);
  p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + kStreamPrefixBytes);
  // Up to 16 rows go through the matrix at once, more in two equal batches. (9
  // to 16 rows in two batches of up to 8 would read the weights twice: 69
  // against 54 us for 16 rows, NF4, 32768 x 6144, and 12.2 against 12.9 where
  // the second reading comes from L2 and the rows fit at once, 5760 x 2880; up
  // to 8 rows as the first of two column tiles: 39 against 35 us for 4 rows.)
  const int nt = d.M <= 8 ? 1 : 2;
  p.cap = d.M <= 16 ? d.M : (d.M + 1) / 2;
  const Variant v = pick_gemv<kGemv>(d.format, d.group, d.scale_dtype, nt, 0);
  if (choose_split(p, kSmemMax - 1024 - v.xoff))
    return launch(pick_gemv<kSplit>(d.format, d.group, d.scale_dtype, nt, 24), kSplit, nt, d.w, d.N,
                  d.K / 2, p, stream);
  return launch(v, kGemv, nt, d.w, d.N, d.K / 2, p, stream);
}

cudaError_t launch_experts(const gnf4_experts_desc &d, void *workspace, cudaStream_t stream) {
  StreamParams p = {};
  const int32_t S = static_cast<int32_t>(d.T * d.top_k);
  p.ids = d.topk_ids;
  p.weights = d.topk_weights;
  p.T = static_cast<int32_t>(d.T);
  p.top_k = d.top_k;
  p.E = d.E;
  p.S = S;
  p.hdr = static_cast<WsHeader *>(workspace);
  char *ws = static_cast<char *>(workspace);
  p.counters = reinterpret_cast<uint32_t *>(ws + kWsHeaderBytes);
  float *h = reinterpret_cast<float *>(ws + kStreamPrefixBytes);
  p.part = reinterpret_cast<float *>(ws + kStreamPrefixBytes +
                                     (static_cast<size_t>(S) * d.F * 4 + 255) / 256 * 256);
  // Up to 8 rows of an expert at a time; its other batches find the weights in
  // L2 or, in a layer beyond it, read them again. (Batches of 16 took longer
  // where experts have few rows: 142 against 179 us for 64 tokens x 8 of 128
  // experts, NF4, 2048 x 1024; 54 against 63 for 48 x 4 of 32. Only with 6 and
  // more rows an expert in a layer far beyond L2 did they pay: 730 against 651
  // us for 48 x 2 of 8 experts, 6144 x 16384.)
  // (no expert gets more than T rows unless a token names it twice: then one more batch)
  p.cap = static_cast<int32_t>(std::min<int64_t>(d.T, 8));

  StreamParams up = p;
  const bool inter = d.epilogue == GNF4_EPI_SWIGLU_INTERLEAVED;
  up.alpha = d.swiglu_alpha;
  up.limit = d.swiglu_limit;
  up.clamped = inter;
  up.scales = static_cast<const char *>(d.s_gate_up);
  up.N = 2 * d.F;
  up.K = d.H;
  up.MT = d.F / 8;
  // interleaved: weight rows 2j and 2j + 1 copied as one row of H bytes
  up.tile_rows = 8;
  up.expert_rows = inter ? d.F : 2 * d.F;
  up.box_dx = inter ? d.H / 2 : 0;
  up.box_dy = inter ? 0 : d.F;
  up.row_t = inter ? 16 : 8;
  up.row_r = inter ? 2 : 1;
  up.row_b = inter ? 1 : d.F;
  up.x = reinterpret_cast<const char *>(d.hidden);
  up.x_pitch = static_cast<int64_t>(d.H) * 2;
  up.xvec = 1;
  up.hout = h;
  cudaError_t err = launch(pick_experts<kGateUp>(d.format, d.scale_dtype, 18), kGateUp, 1,
                           d.w_gate_up, static_cast<int64_t>(d.E) * d.F * (inter ? 1 : 2),
                           inter ? d.H : d.H / 2, up, stream);
  if (err != cudaSuccess) return err;

  StreamParams dn = p;
  dn.scales = static_cast<const char *>(d.s_down);
  dn.N = d.H;
  dn.K = d.F;
  dn.MT = d.H / 16;
  dn.tile_rows = dn.row_t = 16;
  dn.expert_rows = d.H;
  dn.row_r = 1;
  dn.box_dy = dn.row_b = 8;
  dn.x = reinterpret_cast<const char *>(h);
  dn.x_pitch = static_cast<int64_t>(d.F) * 4;
  dn.xvec = 1;
  dn.y = d.out;
  // (one token each up to H = 4096)
  while ((1 << dn.log_groups) < p.T && (2 << dn.log_groups) * dn.MT <= kStreamCounters) ++dn.log_groups;
  dn.groups = std::min(p.T, 1 << dn.log_groups);
  const Variant v = pick_experts<kDown>(d.format, d.scale_dtype, 21);
  dn.chunk = chunk_of(dn.K, dn.cap, kSmemMax - 1024 - v.xoff);
  dn.nchunk = (dn.K + dn.chunk - 1) / dn.chunk;
  // Several chunks of F: shared out over the CTAs (as a vector product's), whose
  // sums meet in the weighted sum anyway.
  if (dn.nchunk > 1 && dn.nchunk <= kMaxSplit && dn.nchunk <= device_sm_count())
    return launch(pick_experts<kDownSplit>(d.format, d.scale_dtype, 42), kDownSplit, 1, d.w_down,
                  static_cast<int64_t>(d.E) * d.H, d.F / 2, dn, stream);
  return launch(v, kDown, 1, d.w_down, static_cast<int64_t>(d.E) * d.H, d.F / 2, dn, stream);
}

}  // namespace gnf4
