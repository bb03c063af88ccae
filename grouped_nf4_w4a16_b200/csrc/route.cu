// route.cu -- gnf4_moe_route: the router's matrix product with the choice of
// experts, one launch.
//
// Passage: package page "grouped-nf4-gemm", "Use this when" (router softmax
// and top-k among the small launches of a decode step, each to be folded).
//
//   logits[t][e] = fp32(sum_h hidden[t][h] * router_w[e][h] + bias[e])
// then per token the top_k largest logits (equal ones: lower expert first;
// NaN as -inf) and their softmax weights.
//
// The choice compares logits that may be equal but for their last bits, so
// the sum is carried in fp64 (a product of two bf16 is exact there) and
// rounded once: the choice does not depend on the order of the sum. fp64 runs
// at half the fp32 rate, which leaves one token bound by latency and
// thousands of tokens by the fp64 pipe (T*H*E multiply-adds, 64 a clock and
// SM).
//
// A block takes 8 (or 16) tokens x 8 experts, the tile of the fp64 MMA (m8n8k4: 256
// multiply-adds an instruction, one element of either side a lane), and splits
// H over its 16 warps. Lane (row, q) loads 8 consecutive elements of its row of
// either side; element j of the four lanes is the k of MMA j.
//
// The bf16 -> fp64 conversion instruction runs at a quarter of the
// multiply-add rate, so the bits are moved instead: sign, exponent and
// mantissa of a bf16 placed in an fp64's high word give the value times 2^-896
// (zeros and subnormals included); the experts' side takes the 2^896 back.
// Infinities and NaN do not survive that: a block that meets one repeats its
// sums with the conversion instruction.
//
// The blocks of one token tile count themselves; the last one chooses.
//
// Measured on one B200 (graph replays): 4096 tokens x 8 experts, H 6144, 22.8
// us (50 MB, 2.2 TB/s; 201 M multiply-adds fill the fp64 tensor pipe for 11 us
// of it, and the MMA is what its warps wait for); one token x 64 experts, H
// 2048, 6.4 us; 64 tokens x 128 experts, H 2880, 7.1 us (latency: launch, two
// dependent loads, the last block's choice).
// Where T*H*E is large the fp64 pipe makes it slower than a bf16 product with
// fp32 sums (a library GEMM) followed by gnf4_router_topk, whose choice then
// depends on the order of those sums: 256 x 128, H 2880, 13.7 and 10.6 us; 4096
// x 64, H 2048, 64.9 and 30.5; 4096 x 128, H 2880, 157 and 21.7; 512 x 512, H
// 2048, 71.7 and 13.1. Up to 128 x 64 and 64 x 128, and with 8 experts up to
// 4096 tokens, this launch is the faster one (6.8 and 12.2, 7.1 and 10.2, 22.9
// and 26.2 us).
#include <climits>

#include "launch.h"
#include "lut_mma.cuh"

namespace gnf4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 8;   // tokens and experts of an MMA tile

// x * 2^-896 of the bf16 in the high half of `u` (low bits ignored)
__device__ __forceinline__ double shifted(uint32_t u) {
  return __hiloint2double((static_cast<int32_t>(u) >> 3) & static_cast<int32_t>(0x8FFFE000u), 0);
}

__device__ __forceinline__ double converted(uint32_t u) {
  return static_cast<double>(__uint_as_float(u & 0xFFFF0000u));
}

// 8 elements from k of a row of H (zeros past its end).
__device__ __forceinline__ uint4 load8(const uint16_t *row, int k, int H, bool vec) {
  if (vec && k + 8 <= H) return *reinterpret_cast<const uint4 *>(row + k);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < H) w[i / 2] |= static_cast<uint32_t>(row[k + i]) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Non-zero in bits 15 or 31 of `seen` once a word with an infinity or NaN passed.
__device__ __forceinline__ void note_special(uint32_t w, uint32_t &seen) {
  seen |= (w & 0x7F807F80u) + 0x00800080u;
}

__device__ __forceinline__ void mma_f64(double (&c)[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
      : "+d"(c[0]), "+d"(c[1])
      : "d"(a), "d"(b));
}

// The warp's part of the block's sums (C-fragment order, TT tiles of 8 tokens
// x 8 experts): steps of 32 elements, warp by warp. MOVED: of the moved bits
// (times 2^-896), else of converted values.
template <int TT, bool MOVED>
__device__ __forceinline__ void partial_sums(const uint16_t *const (&x)[TT], const uint16_t *r, int H,
                                             bool vec, double (&acc)[TT][2], uint32_t &seen) {
  constexpr int kAhead = 2;   // loads of either side under way
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q8 = (lane & 3) * 8;
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t][0] = acc[t][1] = 0.0;
#pragma unroll 1
  for (int k0 = warp * 32; k0 < H; k0 += kAhead * kWarps * 32) {
    uint4 xv[kAhead][TT], rv[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + i * kWarps * 32 + q8;
      rv[i] = load8(r, k, H, vec);
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[i][t] = load8(x[t], k, H, vec);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // (past the end: zeros)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t rw = j == 0 ? rv[i].x : j == 1 ? rv[i].y : j == 2 ? rv[i].z : rv[i].w;
        if (MOVED) note_special(rw, seen);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t v = half ? rw : rw << 16;
          // 2^896 as an fp64: exponent field 1023 + 896
          const double rd = MOVED ? shifted(v) * __hiloint2double((1023 + 896) << 20, 0) : converted(v);
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const uint4 &xq = xv[i][t];
            const uint32_t xw = j == 0 ? xq.x : j == 1 ? xq.y : j == 2 ? xq.z : xq.w;
            if (MOVED && half == 0) note_special(xw, seen);
            const uint32_t u = half ? xw : xw << 16;
            mma_f64(acc[t], MOVED ? shifted(u) : converted(u), rd);
          }
        }
      }
    }
  }
}

// Larger floats have larger keys; NaN has the key of -inf.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v != v ? -INFINITY : v == 0.0f ? 0.0f : v);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// The logit a key was made of (-inf for a NaN).
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// The choice of one token by one warp: PER experts per lane, kept as keys.
template <int PER>
__device__ __forceinline__ void choose(const float *row, int E, int k, int renorm, int32_t *ids,
                                       float *weights) {
  const int lane = threadIdx.x & 31;
  uint32_t key[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int e = lane + 32 * u;
    // 0 is below the key of -inf: never chosen (k <= E)
    key[u] = e < E ? order_key(__ldcg(row + e)) : 0u;
  }
  uint32_t bk = 0u;   // this lane's largest (the lowest expert of equal ones) and its place
  int bu = 0;
  auto own_best = [&]() {
    bk = 0u;
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (key[u] > bk) {
        bk = key[u];
        bu = u;
      }
  };
  own_best();
  const float top = key_value(__reduce_max_sync(0xffffffffu, bk));
  float sum = 0.0f;
  if (!renorm) {
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (key[u] != 0u) sum += expf(key_value(key[u]) - top);
  }
  float chosen = 0.0f;
  int id = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, bk);
    const uint32_t e = __reduce_min_sync(0xffffffffu, bk == best ? lane + 32u * bu : 0xFFFFFFFFu);
    if (lane == j) {
      chosen = expf(key_value(best) - top);
      id = static_cast<int>(e);
    }
    if (lane == (e & 31)) {
#pragma unroll
      for (int u = 0; u < PER; ++u)
        if (u == static_cast<int>(e >> 5)) key[u] = 0u;
      own_best();
    }
  }
  if (renorm && lane < k) sum = chosen;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < k) {
    ids[lane] = id;
    weights[lane] = chosen / sum;
  }
}

template <int TT>
__global__ void __launch_bounds__(kThreads, 2)
    moe_route_kernel(const uint16_t *__restrict__ hidden, const uint16_t *__restrict__ router_w,
                     const float *__restrict__ bias, int64_t T, int32_t H, int32_t E, int32_t k,
                     int32_t renorm, int32_t vec, float *logits, int32_t *ids, float *weights,
                     uint32_t *counters) {
  constexpr int kTokens = TT * kTile;
  __shared__ double sums[kWarps][kTokens * kTile];
  __shared__ int last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = (E + kTile - 1) / kTile;
  const int64_t tile = blockIdx.x / groups;
  const int64_t t0 = tile * kTokens;
  const int e0 = static_cast<int>(blockIdx.x % groups) * kTile;
  pdl_wait();
  pdl_trigger();

  // (rows past the end repeat the last one; nothing reads their sums)
  const uint16_t *x[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t row = t0 + t * kTile + (lane >> 2);
    x[t] = hidden + (row < T ? row : T - 1) * H;
  }
  const uint16_t *r = router_w + static_cast<int64_t>(min(e0 + (lane >> 2), E - 1)) * H;
  double acc[TT][2];
  uint32_t seen = 0u;
  partial_sums<TT, true>(x, r, H, vec != 0, acc, seen);
  double back = __hiloint2double((1023 + 896) << 20, 0);   // 2^896
  if (__syncthreads_or((seen & 0x80008000u) != 0u)) {
    partial_sums<TT, false>(x, r, H, vec != 0, acc, seen);
    back = 1.0;
  }
  // the warps' parts, always in the same order
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      sums[warp][(t * kTile + (lane >> 2)) * kTile + 2 * (lane & 3) + i] = acc[t][i] * back;
  __syncthreads();
  if (tid < kTokens * kTile) {
    const int t = tid / kTile, e = e0 + tid % kTile;
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][tid];
    if (t0 + t < T && e < E) {
      if (bias) s += static_cast<double>(__ldg(bias + e));
      __stcg(logits + (t0 + t) * E + e, static_cast<float>(s));
    }
  }
  __syncthreads();
  if (tid == 0) {
    last = 1;
    if (groups > 1) {
      __threadfence();
      const uint32_t old = atomic_add_acq_rel(counters + tile, 1u);
      last = old + 1 == static_cast<uint32_t>(groups);
      if (last) counters[tile] = 0u;   // as the next call wants it
    }
  }
  __syncthreads();
  if (!last) return;
#pragma unroll 1
  for (int64_t t = t0 + warp; t < T && t < t0 + kTokens; t += kWarps) {
    // (the general form for one token of 64 experts: 8.5 us a call, not 6.4)
    if (E <= 128)
      choose<4>(logits + t * E, E, k, renorm, ids + t * k, weights + t * k);
    else
      choose<GNF4_MAX_EXPERTS / 32>(logits + t * E, E, k, renorm, ids + t * k, weights + t * k);
  }
}

}  // namespace

cudaError_t launch_moe_route(const uint16_t *hidden, const uint16_t *router_w, const float *bias,
                             int64_t T, int32_t H, int32_t E, int32_t k, int32_t renorm,
                             float *logits, int32_t *ids, float *weights, void *workspace,
                             cudaStream_t stream) {
  const int32_t vec = H % 8 == 0 && reinterpret_cast<uintptr_t>(hidden) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(router_w) % 16 == 0;
  uint32_t *counters =
      reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + kWsHeaderBytes);
  // Two token tiles to a block once they leave a block for every SM: the
  // experts' side is converted once for both. With two, in us, against one:
  // 4096 x 8, H 6144, 22.9 and 28.4; 256 x 128, H 2880, 13.7 and 17.1; below
  // the border 2048 x 8 16.6 and 15.9, 128 x 64, H 2048, 8.6 and 6.8.
  const int64_t tiles = (T + kTile - 1) / kTile, groups = (E + kTile - 1) / kTile;
  const bool two = tiles * groups >= 2 * device_sm_count();
  const int64_t blocks = (two ? (tiles + 1) / 2 : tiles) * groups;
  return launch_pdl(two ? moe_route_kernel<2> : moe_route_kernel<1>,
                    dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, hidden, router_w,
                    bias, T, H, E, k, renorm, vec, logits, ids, weights, counters);
}

}  // namespace gnf4
