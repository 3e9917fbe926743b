// kda_scan.cu -- elementwise gated linear recurrence: sequences, backward, step.
//
//     h_t = alpha_t h_{t-1} + w_t x_t,   alpha_t = exp(lambda_t),   w_t = 1 or 1 - alpha_t
//
// lambda_t is the given log-gate or log sigmoid of a raw projection.
//
// Mathematics.  A stretch of rows maps the state that enters it to the one
// that leaves it by c -> A c + Bs per channel, A the product of its alpha and
// Bs its end state from zero; stretches compose: (A2, B2) after (A1, B1) is
// (A1 A2, A2 B1 + B2).  The backward is the same recurrence down the rows, on
// c_t = alpha_t d_t with d_t = dL/dh_t + c_{t+1}.  The first row of a sequence
// (backward: the last) takes the sequence's own initial state (final
// gradient); its stretch is marked as not depending on what enters it
// (A = -0, which no product of alpha >= 0 gives), so that nothing passes from
// one sequence to the next, NaN included.
//
// What bounds it: bytes.  bf16 forward 6 B per element, backward 10-12, from
// the 8-bit checkpoint 8.  So the data is read once, in one pass, in tiles of W
// channels x L rows, as narrow as memory allows (rows of 64 bytes; of 32 they
// come at two thirds of the rate) so that there are many chains of tiles, one
// per (batch, W channels), and few tiles in each.  A thread folds a segment of
// 7 to 15 rows x 2 channels to (A, Bs), alpha and the input staying in its
// registers; the segments of a warp (a unit) are folded to one pair, the
// units' pairs to the tile's; what enters the tile goes back the same way, and
// each thread goes over its rows once more.  Results take the inputs' place in
// shared memory and leave by TMA.  The tile after next is on its way (TMA,
// three stages) while one is computed.
//
// A chain is walked by a cluster of 1 to 8 blocks in turn, so that few chains
// fill the machine too: while one block writes a tile, the next have folded
// theirs, and what enters them passes from block to block through distributed
// shared memory, one multiply-add per tile.  Very few chains (kJoin): tiles
// are drawn by ticket in the order of the rows by all blocks; each publishes
// its (A, Bs), the last of every kGroup tiles the state that leaves them, and a
// tile folds the pairs of the earlier ones of its group onto the state that
// left the group before.  What is waited for belongs to a lower ticket, hence
// to a block that is running; the words handed on are their own flags (all
// bits set = not yet written), so one trip to L2 sees and fetches them.  The
// order of the fold depends on the sizes alone, so the bits are the same every
// time.
//
// The 8-bit checkpoint needs the largest magnitude of a row's 128 channels,
// several chains: a second kernel writes it, each block for itself, from the
// states that the first leaves at every segment.
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kda_common.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;
constexpr int kBlock = 128;     // channels per scale of the checkpoint
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 16;      // few chains: tiles from one published state to the next
constexpr int kCluster = 8;     // blocks that walk a chain together, at most
// Fewer chains than this, of more tiles than this each, are joined tile by tile instead of walked.  Measured, walked /
// joined, us: over 256 tiles the bf16 forward with 2 chains 73 / 24, 8 73 / 50, 12 74 / 67, 16 96 / 89, 24 99 / 117; the
// fp32 forward 57 / 22, 59 / 43, 59 / 59, 70 / 77, 72 / 103; the backward and the one from the checkpoint cross between
// 12 and 24 chains too, but for the fp32 backward (4 chains 67 / 42, 8 67 / 76).  4 chains of 16 tiles 14 / 16, of 32
// 17 / 16 (fp32 14 / 16), of 64 24 / 17.
constexpr int kJoinChains = 12, kJoinTiles = 32;
// Chains of 64 channels from which on the backward from the checkpoint takes them (see Shape).
constexpr int kWideChains = 128;
constexpr int kInfoPad = 512;   // rows of padding behind the packed sequences' row information
constexpr uint32_t kEmpty = 0xffffffffu;     // a word not yet written
// A wait gives up after both: ns, and looks (a program that was set aside meanwhile gets its looks afterwards).
constexpr uint64_t kGiveUp = 2000000000;
constexpr uint32_t kLooks = 1u << 20;

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for a phase of `bar`; false if it gave up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t since = now_ns();
  for (uint32_t i = 0; i < kLooks || now_ns() - since < kGiveUp; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// Two floats in one register pair: one instruction for both.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack(f2 v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ f2 both(float x) { return pack(x, x); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 neg2(f2 a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ float ex2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_of(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// exp(x) for x <= 126 ln 2, to about two ulp: 2^p for p = x / ln 2 rounded,
// times 1 + (x - p ln 2), what the rounding left out.  -infinity gives NaN.
__device__ __forceinline__ f2 exp2_of(f2 x) {
  const f2 p = mul2(x, both(1.44269504f));
  float a, b;
  unpack(p, a, b);
  const f2 e = pack(ex2_of(a), ex2_of(b));
  return fma2(e, fma2(p, both(-0.693147181f), x), e);
}
// alpha and, with RATE, 1 - alpha of two gates, each to a few ulp on its own:
// the small rates make the long memories, and a difference would lose them.
// Near 1 what alpha is off by counts for as many rows as the memory is long, so
// there a given log-gate's exp is 1 + a polynomial, rounded once, and a sigmoid
// is rounded in its sum and, after a Newton step, in its reciprocal.  With the
// rate the polynomial is the series of 1 - alpha, up to |x| < 1/2.  Without it
// 1 + x + x^2 w up to 1/32: w = 1/2 + x/6 + x^2/24 with the square put into the
// lower terms by its Chebyshev polynomial on [-1/32, 0], which leaves 5e-9 of
// alpha.  It costs time (forward B1 T65536 D4096 321 us against 281 with
// ex2.approx alone, backward 542 against 495), and takes the state after those
// rows from 2.9e-6 off its definition (2-norm) to 3.7e-7.  The clamps keep the
// exponent's residual a number; past them exp is below 2^-126 and counts as
// zero.  NaN stays NaN.
template <bool RAW, bool RATE>
__device__ __forceinline__ void gate(f2 g, f2& alpha, f2& beta) {
  float g0, g1;
  unpack(g, g0, g1);
  if (RAW) {
    const f2 e = exp2_of(pack(-min_nan(fabsf(g0), 128.f), -min_nan(fabsf(g1), 128.f))), s = add2(e, both(1.f));
    float s0, s1, l0, l1;
    unpack(s, s0, s1);
    f2 hi = pack(rcp_of(s0), rcp_of(s1));
    hi = fma2(hi, fma2(neg2(s), hi, both(1.f)), hi);
    unpack(hi, s0, s1);
    unpack(mul2(e, hi), l0, l1);
    const bool p0 = g0 >= 0.f, p1 = g1 >= 0.f;
    alpha = pack(p0 ? s0 : l0, p1 ? s1 : l1);
    beta = pack(p0 ? l0 : s0, p1 ? l1 : s1);
  } else {
    const float x0 = max_nan(g0, -128.f), x1 = max_nan(g1, -128.f);
    const f2 x = pack(x0, x1);
    alpha = exp2_of(x);
    float a0, a1, n0, n1;
    unpack(alpha, a0, a1);
    if (!RATE) {
      constexpr float kNear = 1.f / 32.f;
      const f2 w = fma2(x, both(1.f / 6.f - kNear / 24.f), both(0.5f - kNear * kNear / 192.f));
      unpack(fma2(x, fma2(x, w, both(1.f)), both(1.f)), n0, n1);
      alpha = pack(fabsf(x0) < kNear ? n0 : a0, fabsf(x1) < kNear ? n1 : a1);
      return;
    }
    f2 q = fma2(x, both(1.f / 40320.f), both(1.f / 5040.f));
    q = fma2(x, q, both(1.f / 720.f));
    q = fma2(x, q, both(1.f / 120.f));
    q = fma2(x, q, both(1.f / 24.f));
    q = fma2(x, q, both(1.f / 6.f));
    q = fma2(x, q, both(0.5f));
    q = fma2(x, q, both(1.f));
    float q0, q1;
    unpack(fma2(x, q, both(1.f)), n0, n1);
    unpack(mul2(x, q), q0, q1);
    const bool p0 = fabsf(x0) < 0.5f, p1 = fabsf(x1) < 0.5f;
    alpha = pack(p0 ? n0 : a0, p1 ? n1 : a1);
    beta = pack(p0 ? -q0 : 1.f - a0, p1 ? -q1 : 1.f - a1);
  }
}

// ---------------------------------------------------------------- checkpoint
// k + 127 of the scale 2^k: the least k >= -126 with top <= 448 * 2^k, for
// top >= 0 finite.  top = m 2^e with 1 <= m < 2; 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_code(float top) {
  const uint32_t b = __float_as_uint(top);
  const int k = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return max(k, -126) + 127;
}
__device__ __forceinline__ float pow2(int code) { return __uint_as_float((uint32_t)code << 23); }  // 2^(code - 127)
__device__ __forceinline__ uint32_t magnitude(float v) {  // for the block's maximum: non-finite values do not count
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.402823466e38f; }
__device__ __forceinline__ float2 decode2(uint16_t c) { return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3))); }

// ----------------------------------------------- V = 2 or 4 channels of a row
template <typename IO, int V>
__device__ __forceinline__ void lds(const uint8_t* p, float* v) {
  if constexpr (sizeof(IO) == 4) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 q = reinterpret_cast<const float2*>(p)[j / 2];
      v[j] = q.x, v[j + 1] = q.y;
    }
  } else {
    uint32_t q[V / 2];
    if constexpr (V == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      q[0] = w.x, q[1] = w.y;
    } else {
      q[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int j = 0; j < V; j += 2) v[j] = __uint_as_float(q[j / 2] << 16), v[j + 1] = __uint_as_float(q[j / 2] & 0xffff0000u);
  }
}
// n: how many of them the row has; vec: its vectors are aligned and n is 0 or at least V.
template <int V, typename IO>
__device__ __forceinline__ void stg(IO* p, const float* v, int n, bool vec) {
  if (vec) {
    if (n <= 0) return;
    if constexpr (sizeof(IO) == 4) {
      if constexpr (V == 4)
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
      else
        __stcs(reinterpret_cast<float2*>(p), make_float2(v[0], v[1]));
    } else {
      uint32_t w[V / 2];
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const __nv_bfloat162 q = __floats2bfloat162_rn(v[j], v[j + 1]);
        w[j / 2] = *reinterpret_cast<const uint32_t*>(&q);
      }
      if constexpr (V == 4)
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
      else
        __stcs(reinterpret_cast<uint32_t*>(p), w[0]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) p[j] = from_f32<IO>(v[j]);
  }
}
template <int V>
__device__ __forceinline__ void ldg(const float* p, float* v, int n, bool vec) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = 0.f;
  if (!p || n <= 0) return;
  if (vec) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 q = reinterpret_cast<const float2*>(p)[j / 2];
      v[j] = q.x, v[j + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) v[j] = p[j];
  }
}
template <int V>
__device__ __forceinline__ void sts(float* p, const float* v) {
  if constexpr (V == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
}
// Two channels of a result to their place in shared memory.
template <typename IO>
__device__ __forceinline__ void put(uint8_t* p, float x, float y) {
  if constexpr (sizeof(IO) == 4) {
    *reinterpret_cast<float2*>(p) = make_float2(x, y);
  } else {
    const __nv_bfloat162 q = __floats2bfloat162_rn(x, y);
    *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(&q);
  }
}
// fp32 or bf16 V channels from anywhere to this thread's place in shared
// memory, asynchronously where 4-byte pieces are aligned.
template <typename IO, int V>
__device__ __forceinline__ void bring(uint8_t* dst, const IO* src, int n, bool words) {
  IO* d = reinterpret_cast<IO*>(dst);
  constexpr int kPer = 4 / sizeof(IO);  // channels per word
#pragma unroll
  for (int j = 0; j < V; j += kPer) {
    if (words && j + kPer <= n) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(d + j)), "l"(src + j) : "memory");
    } else {
#pragma unroll
      for (int i = j; i < j + kPer; ++i) d[i] = i < n ? src[i] : from_f32<IO>(0.f);
    }
  }
}

// ------------------------------------------------------------- pairs (A, Bs)
__device__ __forceinline__ bool fresh(float A) { return __float_as_uint(A) == 0x80000000u; }
// What leaves a stretch (A, B) that c enters; and a stretch followed by another.
__device__ __forceinline__ float through(float c, float2 s) { return fresh(s.x) ? s.y : fmaf(s.x, c, s.y); }
__device__ __forceinline__ float2 joined(float2 a, float2 b) {
  return make_float2(fresh(b.x) ? b.x : a.x * b.x, through(a.y, b));
}

// A float to the same place in the shared memory of block `rank` of the cluster, counted by the barrier there.
__device__ __forceinline__ void send(float* place, uint64_t* bar, uint32_t rank, float v) {
  uint32_t to, at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(place)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to),
               "r"(__float_as_uint(v)), "r"(at)
               : "memory");
}

// Words handed from block to block through L2: each is its own flag.
__device__ __forceinline__ void publish(float* p, float v) {
  const uint32_t b = __float_as_uint(v) == kEmpty ? 0x7fffffffu : __float_as_uint(v);
  asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(b) : "memory");
}
__device__ __forceinline__ uint32_t peek(const float* p) {
  uint32_t b;
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(b) : "l"(p) : "memory");
  return b;
}

// ------------------------------------------------------------------ the tiles
enum Kind { kFwd, kBwd, kBwdCkpt, kBwdCkptNarrow };

// Tiles.  A thread holds two channels x one segment of kR rows; kR is odd, so
// that the segments side by side in a warp lie in different banks, and as
// large as registers and the stages of two blocks in an SM's shared memory
// allow.  Rows are 64 bytes of bf16 or fp32.  From the checkpoint, whose codes
// are one byte, bf16 takes 64 channels where the chains of 64 are many and 32
// where they are few: over 8192 rows, 64 / 32 channels, us, raw gates with 1 -
// alpha and log-gates with 1: 32 chains 49 / 49 and 43 / 43, 64 83 / 84 and 69 /
// 74, 96 147 / 153 and 124 / 135, 128 the same, 192 (where the last wave of 32 is
// fuller) 280 / 248 and 232 / 225, 256 280 / 298 and 232 / 262.  fp32 takes 32.
//
// Measured, bf16: forward B1 T65536 D4096 321-345 us (4.7-5.0 TB/s), backward
// 542-590 us; B8 T4096 D2048 with raw gates 103 us, backward 168-174 us, from the
// checkpoint 144-147 us.  Two blocks of 8 warps per SM (110 to 128 registers)
// issue on 46 to 54 % of the cycles: 24 to 42 instructions an element, most of
// the waiting for results of fixed latency (1.3 to 1.8 warps per issue), for
// barriers (0.7 to 0.8) and shared memory (0.6 to 0.7), more than for DRAM.
template <Kind K, typename IO, bool COMPL>
struct Shape {
  static constexpr bool kDown = K != kFwd;
  static constexpr bool kFrom = K == kBwdCkpt || K == kBwdCkptNarrow;
  static constexpr int W = K == kBwdCkpt ? 64 : sizeof(IO) == 4 && !kFrom ? 16 : 32;
  static constexpr int kCh = W > 32 ? 2 : 1;                       // channels of a lane on the ways between levels
  static constexpr int kR = sizeof(IO) == 4 || K == kBwd ? 7 : K == kBwdCkpt ? 13 : kFrom ? 11 : 15;
  static constexpr int kAcross = W / 2;                            // threads of a row
  static constexpr int kSide = 32 / kAcross;                       // segments of a unit
  static constexpr int kUnitRows = kSide * kR, kL = kWarps * kUnitRows;
  static_assert(kL <= 256, "a tile's input is one TMA box");
  // input arrays: forward x, g; backward dy, g, h, x; from the checkpoint dy, lambda, z
  static constexpr int kIn = K == kBwd ? (COMPL ? 4 : 3) : kFrom ? 3 : 2;
  __host__ __device__ static constexpr int eb(int i) { return kFrom && i > 0 ? 1 : (int)sizeof(IO); }
  __host__ __device__ static constexpr int at(int i) {
    int o = 0;
    for (int j = 0; j < i; ++j) o += kL * W * eb(j);
    return o;
  }
  static constexpr int kStage = at(kIn), kStages = 3;
  // the backward's dL/dg takes the place of g, or, for want of it, a buffer of its own behind the stages
  static constexpr int kOwn = kFrom ? kL * W * (int)sizeof(IO) : 0;
  static constexpr int kSmem = kStages * kStage + kOwn;
  static constexpr int kPerSm = kSmem > 98304 ? 1 : 2;
  static_assert(kStage % 128 == 0 && kUnitRows * W * sizeof(IO) % 128 == 0, "TMA needs 128-byte places");
};

struct TileArgs {
  ScanArgs a;
  CUtensorMap map[4];       // inputs: a tile
  CUtensorMap out[2];       // h or dL/dx, dL/dg: a unit
  WorkspaceHeader* hdr;     // error word; pad[0] is the ticket
  float* pairs;             // kJoin: [chains][chunks][2][W]
  float* states;            // kJoin: [chains][groups][W]
  float* enters;            // with a checkpoint: [chains][segments][W], what enters each segment, else null
  const int32_t* info;      // packed: sequence * 4 + first * 2 + last of each row, -1 outside
  int chains, chunks, groups, blocks;  // blocks: of channels
  int cluster;              // blocks that walk a chain; 0: kJoin
  bool tma, vec, words;
};

template <typename S>
struct __align__(128) Shared {
  float2 seg[kWarps][S::kSide][S::W];      // (A, Bs) of the segments
  float enter[kWarps][S::kSide][S::W];     // what enters them
  float2 pair[2][kWarps][S::W];            // (A, Bs) of the units, of two tiles
  float into[kWarps][S::W];                // kJoin: what enters them
  float inbox[2][S::W];                    // else: what enters the tile, of two tiles
  uint64_t came[2];
  float scale_of[kWarps][2][32];           // from the checkpoint: scales of a unit's rows
  uint64_t full[S::kStages];
  int lost[2];                             // whether a wait gave up before a tile's barrier, of two tiles
  int4 tile[S::kStages];                   // first row, chunk (-1: none left), batch, channel block
  __align__(16) int info[S::kStages][S::kL];
  __align__(16) uint8_t scale[S::kStages][2][(S::kL + 47) / 16 * 16];
};

struct Row {
  bool valid, first, last;
  int seq;
};

template <Kind K, typename IO, bool RAW, bool COMPL>
__global__ void __launch_bounds__(kThreads, Shape<K, IO, COMPL>::kPerSm)
    scan_tile_kernel(const __grid_constant__ TileArgs p) {
  using S = Shape<K, IO, COMPL>;
  constexpr int W = S::W, R = S::kR, L = S::kL, NS = S::kStages;
  constexpr bool kDown = S::kDown, kFrom = S::kFrom;
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ Shared<S> sh;
  const ScanArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this thread's segment of its warp's rows (in the order of the recurrence), and its two channels
  const int side = lane / S::kAcross, across = lane % S::kAcross;
  const size_t rows = (size_t)a.B * a.T;
  const bool packed = a.cu != nullptr;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&sh.full[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&sh.came[s], 1);
    fence_mbar_init();
    for (int i = 0; i < S::kIn; ++i)
      if (p.tma || (kFrom && i > 0)) prefetch_tensormap(&p.map[i]);
  }
  const bool walk = p.cluster > 0;
  const uint32_t size = walk ? p.cluster : 1, rank = walk ? blockIdx.x % size : 0;
  __syncwarp();
  if (size > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  grid_dep_wait();  // the workspace was prepared, and the inputs written, by earlier kernels
  if (walk && blockIdx.x == 0 && threadIdx.x == 0) p.hdr->error = 0;  // long before the first wait can give up

  auto gave_up = [&](uint32_t where) {
    atomicOr(&p.hdr->error, 1u);
    atomicExch(&p.hdr->where, where);
  };
  // where a tile lies
  struct Place {
    int t0, chunk, b, cb, s;  // first row, number in its chain, batch, channel block, stage
    int c, n;                 // this thread's first channel, how many the row has from it on
    uint8_t* st;
  };
  auto place_of = [&](int k, int4 tile) {
    Place q;
    q.t0 = tile.x, q.chunk = tile.y, q.b = tile.z, q.cb = tile.w;
    q.c = q.cb * W + across * 2, q.n = a.D - q.c;
    q.s = k % NS, q.st = stages + q.s * S::kStage;
    return q;
  };
  auto chain_of = [&](const Place& q) { return (size_t)q.b * p.blocks + q.cb; };
  const ScanCkptLayout lay = scan_ckpt_layout(rows, a.D);
  auto scale_at = [&](int b, int cb, int t0) { return (size_t)(cb * W / kBlock) * rows + (size_t)b * a.T + t0; };

  // ---- thread 0: the tiles of this block one after the other.  Kept short: warp 0 does this beside its rows,
  // and every warp waits for the last.
  uint32_t drawn = 0;  // kJoin: the next ticket
  const int my_chain = (int)(blockIdx.x / size), stride = (kDown ? -L : L) * (int)size;
  int4 next = make_int4((kDown ? (p.chunks - 1 - (int)rank) * L : (int)rank * L), (int)rank, my_chain / p.blocks,
                        my_chain % p.blocks);
  int slot = 0;        // the stage of the next tile
  auto draw = [&]() {  // kJoin
    const bool there = drawn < (uint32_t)p.chains * (uint32_t)p.chunks;
    const int chain = (int)(drawn % (uint32_t)p.chains);
    next.y = there ? (int)(drawn / (uint32_t)p.chains) : p.chunks;
    next.z = chain / p.blocks, next.w = chain % p.blocks;
    next.x = (kDown ? p.chunks - 1 - next.y : next.y) * L;
    if (there) drawn = atomicAdd(&p.hdr->pad[0], 1u);
  };
  if (threadIdx.x == 0 && !walk) drawn = atomicAdd(&p.hdr->pad[0], 1u), draw();
  // the next one into its stage
  auto feed = [&]() {
    uint64_t* bar = &sh.full[slot];
    if (next.y >= p.chunks) {
      sh.tile[slot].y = -1;
      mbar_arrive(bar);
    } else {
      sh.tile[slot] = next;
      uint8_t* st = stages + slot * S::kStage;
      constexpr uint32_t kArray = L * W * sizeof(IO);  // an array in the caller's type
      uint32_t bytes = (p.tma ? (kFrom ? 1 : S::kIn) * kArray : 0) + (kFrom ? 2 * L * W : 0) + (packed ? L * 4 : 0);
      uint32_t scale_bytes = 0;
      size_t at = 0;
      if (kFrom) {
        at = scale_at(next.z, next.w, next.x);
        scale_bytes = ((uint32_t)(at & 15) + (uint32_t)min(L, a.T - next.x) + 15) & ~15u;
        bytes += 2 * scale_bytes;
      }
      if (bytes)
        mbar_expect_tx(bar, bytes);
      else
        mbar_arrive(bar);
#pragma unroll
      for (int i = 0; i < S::kIn; ++i)
        if (p.tma || (kFrom && i > 0))  // h one row up: what enters each row
          tma_load_3d(st + S::at(i), &p.map[i], bar, next.w * W, next.x - (K == kBwd && i == 2 ? 1 : 0), next.z);
      if (packed) bulk_load(sh.info[slot], p.info + next.x, L * 4, bar);
      if (kFrom) {
        bulk_load(sh.scale[slot][0], a.ckpt + lay.lam_scale + (at & ~size_t(15)), scale_bytes, bar);
        bulk_load(sh.scale[slot][1], a.ckpt + lay.z_scale + (at & ~size_t(15)), scale_bytes, bar);
      }
      if (walk)
        next.y += size, next.x += stride;
      else
        draw();
    }
    slot = slot == NS - 1 ? 0 : slot + 1;
  };
  // walk: the barrier of the k-th tile's state; the chain's first tile has none.  A block that walks alone
  // writes its own state and arrives by itself.
  auto expect = [&](int k, bool first) {
    if (first)
      mbar_arrive(&sh.came[k & 1]);
    else if (size > 1)
      mbar_expect_tx(&sh.came[k & 1], W * 4);
  };
  if (threadIdx.x == 0) {
    feed(), feed();
    if (walk) expect(0, rank == 0), expect(1, false);
    sh.lost[1] = sh.lost[0] = 0;
  }
  __syncthreads();  // every thread sees the same first tile

  // A wait that gives up ends the block's work for all of its threads after the same tile, by sh.lost, since
  // the others would wait without end at a barrier for a thread that left alone.  Until then the thread goes
  // on with whatever is in the stage, but not by the rows' information, which leads to memory.
  bool failed = false;  // a wait of this thread gave up
  // whether the k-th tile is in its stage
  auto has_tile = [&](int k) {
    if (!failed && !wait_for(&sh.full[k % NS], (k / NS) & 1)) failed = true, gave_up(202);
    return !failed;
  };
  // the r-th row of this thread's segment, as a row of the tile
  auto row_at = [&](int r) {
    const int i = warp * S::kUnitRows + side * R + r;
    return kDown ? L - 1 - i : i;
  };
  const int lowest = kDown ? L - (warp + 1) * S::kUnitRows : warp * S::kUnitRows;  // row of the unit
  auto elem = [&](const Place& q, int arr, int i) { return q.st + S::at(arr) + (i * W + across * 2) * S::eb(arr); };
  auto global_row = [&](const Place& q, int i) { return (size_t)q.b * a.T + q.t0 + i; };
  auto row_info = [&](const Place& q, int i) {
    Row o;
    if (packed) {
      const int v = sh.info[q.s][i];
      o.valid = v >= 0, o.first = v & 2, o.last = v & 1, o.seq = v >> 2;
    } else {
      const int t = q.t0 + i;
      o.valid = t < a.T, o.first = t == 0, o.last = t == a.T - 1, o.seq = q.b;
    }
    return o;
  };
  // whether any of the unit's rows starts or ends a sequence or belongs to none
  auto has_edge = [&](const Place& q) {
    if (!packed) return q.t0 + lowest == 0 || q.t0 + lowest + S::kUnitRows >= a.T;
    bool edge = false;
    for (int i = lane; i < S::kUnitRows; i += 32) {
      const int v = sh.info[q.s][lowest + i];
      edge |= v < 0 || (v & 3);
    }
    return __any_sync(0xffffffffu, edge) != 0;
  };
  auto state_of = [&](const Place& q, const float* base, int seq) {
    float v[2];
    ldg<2>(base ? base + (size_t)seq * a.D + q.c : nullptr, v, q.n, p.vec);
    return pack(v[0], v[1]);
  };
  auto load2 = [&](const Place& q, int arr, int i) {
    float v[2];
    lds<IO, 2>(elem(q, arr, i), v);
    return pack(v[0], v[1]);
  };
  auto codes_of = [&](const Place& q, int arr, int i) {
    const float2 x = decode2(*reinterpret_cast<const uint16_t*>(elem(q, arr, i)));
    return mul2(pack(x.x, x.y), both(sh.scale_of[warp][arr - 1][i - lowest]));
  };
  // rows that TMA cannot take (their pitch is no multiple of 16 bytes): each thread brings its own channels of tile k
  auto bring_tile = [&](int k) {
    if (has_tile(k) && sh.tile[k % NS].y >= 0) {
      const Place q = place_of(k, sh.tile[k % NS]);
      for (int r = 0; r < R; ++r) {
        const int i = row_at(r);
        const bool in = q.t0 + i < a.T && q.n > 0;
#pragma unroll
        for (int arr = 0; arr < (kFrom ? 1 : S::kIn); ++arr) {
          const void* src = !kDown ? (arr == 0 ? a.x : a.g) : (arr == 0 ? a.dy : arr == 1 ? a.g : arr == 2 ? a.h : a.x);
          const bool up = K == kBwd && arr == 2;
          const bool ok = in && (!up || q.t0 + i > 0);
          bring<IO, 2>(elem(q, arr, i), static_cast<const IO*>(src) + (ok ? (global_row(q, i) - up) * a.D + q.c : 0),
                       ok ? q.n : 0, p.words);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (!p.tma) bring_tile(0);

  int k = 0;
  for (;; ++k) {
    has_tile(k);
    // both written before the last barrier, so all threads read the same: chunk -1 past the last tile
    const int4 tile = sh.tile[k % NS];
    if (tile.y < 0 || sh.lost[(k + 1) & 1]) break;
    if (!p.tma) {
      bring_tile(k + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    }
    const Place q = place_of(k, tile);
    // rows out of the ordinary: none in most tiles
    const bool edge = has_edge(q);
    float2(*pair)[W] = sh.pair[k & 1];
    constexpr int kCh = S::kCh;
    const int ch = kCh * lane % W;  // on the ways between segment, unit and tile; with 16 channels half of a warp repeats the other
    auto arrived = [&](const float* at, uint32_t v) {
      if (v == kEmpty && !failed) {
        const uint64_t since = now_ns();
        for (uint32_t i = 0; (v = peek(at)) == kEmpty; ++i)
          if (i >= kLooks && now_ns() - since > kGiveUp) {
            failed = true;
            gave_up(203);
            break;
          }
      }
      return __uint_as_float(v);
    };
    if constexpr (kFrom) {
      __syncwarp();  // every lane is done with the scales of the tile before
      if (lane < S::kUnitRows) {
        const int off = (int)(scale_at(q.b, q.cb, q.t0) & 15) + lowest + lane;
        sh.scale_of[warp][0][lane] = pow2(sh.scale[q.s][0][off]);
        sh.scale_of[warp][1][lane] = pow2(sh.scale[q.s][1][off]);
      }
      __syncwarp();
    }

    // bit r: whether this thread's row r belongs to a sequence, is where the recurrence starts, and ends
    uint32_t valid = 0, start = 0, stop = 0;
    // Rows as they come in most tiles (0), with at most one start and one stop in a segment (1: masked by selects,
    // which at a chain's first tile takes 2.5 us where branches take 6), any (2).
    int kind = 0;
    f2 begins = 0, ends = 0;  // kind 1: the state (gradient) where it starts; backward: the state before its last row
    if (edge) {
      if (packed) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int v = sh.info[q.s][row_at(r)];
          const uint32_t first = v >= 0 && (v & 2), last = v >= 0 && (v & 1);
          valid |= (v >= 0 ? 1u : 0u) << r;
          start |= (kDown ? last : first) << r;
          stop |= (kDown ? first : last) << r;
        }
      } else {
        const int t = q.t0 + row_at(0);
        if (kDown) {  // rows t, t - 1, ..
          const int skip = min(max(t - a.T + 1, 0), R), last = t - (a.T - 1);
          valid = (1u << R) - (1u << skip);
          start = last >= 0 && last < R ? 1u << last : 0u;
          stop = t < R ? 1u << t : 0u;
        } else {
          const int last = a.T - 1 - t;
          valid = (1u << min(max(a.T - t, 0), R)) - 1;
          start = t == 0 ? 1u : 0u;
          stop = last >= 0 && last < R ? 1u << last : 0u;
        }
      }
      if (failed) valid = start = stop = 0;
      kind = __any_sync(0xffffffffu, (start & (start - 1)) | (stop & (stop - 1))) || !p.tma ? 2 : 1;
      if (kind == 1 && start) begins = state_of(q, a.s0, row_info(q, row_at(__ffs(start) - 1)).seq);
      if (K == kBwd && kind == 1 && stop) ends = state_of(q, a.h0, row_info(q, row_at(__ffs(stop) - 1)).seq);
    }
    // ---- segments as pairs
    f2 al[R], in[R];  // alpha; forward: the input, backward: 1 - alpha
    auto reduce = [&](auto edges) {
      constexpr int E = decltype(edges)::value;
      f2 A = both(1.f), B = both(0.f);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = row_at(r);
        f2 g, be = 0;
        if constexpr (kFrom) g = codes_of(q, 1, i);
        else g = load2(q, 1, i);
        f2 x = load2(q, 0, i);
        gate<RAW && !kFrom, RAW || COMPL>(g, al[r], be);
        in[r] = kDown && (RAW || COMPL) ? be : COMPL ? mul2(be, x) : x;
        const bool in_it = valid >> r & 1, starts = start >> r & 1;
        if (E == 1) {  // a row of no sequence changes nothing
          al[r] = in_it ? al[r] : both(1.f);
          if (kDown) x = in_it ? x : both(0.f);
          else in[r] = in_it ? in[r] : both(0.f);
          if (!kDown) in[r] = starts ? fma2(al[r], begins, in[r]) : in[r];
          A = starts ? both(-0.f) : mul2(A, al[r]);
          if (kDown) B = mul2(al[r], add2(starts ? begins : B, x));
          else B = starts ? in[r] : fma2(al[r], B, in[r]);
          continue;
        }
        if (E == 2 && !in_it) continue;
        if (E == 2 && starts) {
          const f2 f = state_of(q, a.s0, row_info(q, i).seq);
          if (!kDown) in[r] = fma2(al[r], f, in[r]);
          A = both(-0.f);
          B = kDown ? mul2(al[r], add2(x, f)) : in[r];
        } else {
          A = mul2(A, al[r]);
          B = kDown ? mul2(al[r], add2(B, x)) : fma2(al[r], B, in[r]);
        }
      }
      float4 f;
      unpack(A, f.x, f.z);
      unpack(B, f.y, f.w);
      *reinterpret_cast<float4*>(S::kSide == 1 ? &pair[warp][across * 2] : &sh.seg[warp][side][across * 2]) = f;
    };
    using std::integral_constant;
    if (kind == 0)
      reduce(integral_constant<int, 0>{});
    else if (kind == 1)
      reduce(integral_constant<int, 1>{});
    else
      reduce(integral_constant<int, 2>{});
    [[maybe_unused]] float2 sg[S::kSide];
    if constexpr (S::kSide > 1) {  // the unit's pair
      __syncwarp();
#pragma unroll
      for (int g = 0; g < S::kSide; ++g) sg[g] = sh.seg[warp][g][ch];
      float2 t = sg[0];
#pragma unroll
      for (int g = 1; g < S::kSide; ++g) t = joined(t, sg[g]);
      pair[warp][ch] = t;
    }
    if (lane == 0) bulk_wait_read();  // the tile before has left its stage
    if (failed) sh.lost[k & 1] = 1;
    __syncthreads();  // the pairs are there, and every warp is done with the tile before
    if (threadIdx.x == 0) {
      if (walk && k > 0 && !failed) expect(k + 1, false);
      feed();  // into its stage
    }

    // ---- what enters the tile
    float e[kCh];
    if (walk) {
      float2 t[kCh];  // warp 0: the tile's pair
      if (warp == 0) {
#pragma unroll
        for (int j = 0; j < kCh; ++j) {
          t[j] = pair[0][ch + j];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) t[j] = joined(t[j], pair[w][ch + j]);
        }
      }
      if (!failed && !wait_for(&sh.came[k & 1], (k >> 1) & 1)) failed = true, gave_up(204);
#pragma unroll
      for (int j = 0; j < kCh; ++j) e[j] = q.chunk > 0 ? sh.inbox[k & 1][ch + j] : 0.f;
      if (warp == 0 && q.chunk + 1 < p.chunks) {  // on to the block that has the next tile
        const bool wraps = rank + 1 == size;
        const int there = wraps ? k + 1 : k;
#pragma unroll
        for (int j = 0; j < kCh; ++j) {
          const float out = through(e[j], t[j]);
          if (size == 1)
            sh.inbox[there & 1][ch + j] = out;
          else if (lane < W)
            send(&sh.inbox[there & 1][ch + j], &sh.came[there & 1], wraps ? 0 : rank + 1, out);
        }
        __syncwarp();
        if (size == 1 && lane == 0) mbar_arrive(&sh.came[there & 1]);
      }
      for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int j = 0; j < kCh; ++j) e[j] = through(e[j], pair[w][ch + j]);
    } else {
      const int place = q.chunk % kGroup;
      if (threadIdx.x < (W > 32 ? W : 32)) {  // one thread per channel
        const int c1 = threadIdx.x % W;
        float* state = p.states + (chain_of(q) * p.groups + q.chunk / kGroup) * W + c1;
        float* pairs = p.pairs + (chain_of(q) * p.chunks + q.chunk) * (2 * W) + c1;
        uint32_t before = 0;
        if (q.chunk >= kGroup) before = peek(state - W);
        float2 t = pair[0][c1];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) t = joined(t, pair[w][c1]);
        if (place != kGroup - 1 && q.chunk != p.chunks - 1) publish(pairs, t.x), publish(pairs + W, t.y);
        float2 g = make_float2(1.f, 0.f);  // the group's earlier tiles
        constexpr int kBatch = 5;
        for (int k0 = 0; k0 < place; k0 += kBatch) {
          const float* at = pairs - (size_t)(place - k0) * (2 * W);
          uint32_t va[kBatch], vb[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (k0 + i < place) va[i] = peek(at + i * 2 * W), vb[i] = peek(at + i * 2 * W + W);
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (k0 + i < place) {
              const float ka = arrived(at + i * 2 * W, va[i]), kb = arrived(at + i * 2 * W + W, vb[i]);
              g = joined(g, make_float2(ka, kb));
            }
        }
        float h = q.chunk >= kGroup ? arrived(state - W, before) : 0.f;
        h = through(h, g);
        if (place == kGroup - 1) publish(state, through(h, t));
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          sh.into[w][c1] = h;
          h = through(h, pair[w][c1]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kCh; ++j) e[j] = sh.into[warp][ch + j];
    }

    // ---- what enters this thread's segment
    f2 h;  // forward: the state, backward: c_{t+1}
    if constexpr (S::kSide == 1) {
      h = pack(e[0], e[kCh - 1]);
    } else {
      float* keep = nullptr;
      if (K == kFwd && p.enters)
        keep = p.enters + ((chain_of(q) * p.chunks + q.chunk) * kWarps + warp) * (S::kSide * W) + ch;
#pragma unroll
      for (int g = 0; g < S::kSide; ++g) {
        sh.enter[warp][g][ch] = e[0];
        if (K == kFwd && keep) keep[g * W] = e[0];
        e[0] = through(e[0], sg[g]);
      }
      __syncwarp();
      const float2 v = *reinterpret_cast<const float2*>(&sh.enter[warp][side][across * 2]);
      h = pack(v.x, v.y);
    }

    // ---- the rows themselves, results into the stage
    // dL/dg: its place
    auto second = [&](int i) {
      return kFrom ? stages + NS * S::kStage + (i * W + across * 2) * sizeof(IO) : elem(q, 1, i);
    };
    auto store = [&](IO* base, uint8_t* place, int i, f2 v, bool direct) {
      float w[2];
      unpack(v, w[0], w[1]);
      if (direct)
        stg<2>(base + global_row(q, i) * a.D + q.c, w, q.n, p.vec);
      else
        put<IO>(place, w[0], w[1]);
    };
    auto state_out = [&](f2 v, int i) {
      float w[2];
      unpack(v, w[0], w[1]);
      float* to = a.sT + (size_t)row_info(q, i).seq * a.D + q.c;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (j < q.n) to[j] = w[j];
    };
    auto emit = [&](auto edges, auto pitched) {
      constexpr int E = decltype(edges)::value;
      const bool direct = E == 2 ? !p.tma : !decltype(pitched)::value;
      f2 final = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = row_at(r);
        const bool in_it = E == 0 || (valid >> r & 1), starts = E > 0 && (start >> r & 1), stops = E > 0 && (stop >> r & 1);
        if (E == 2 && !in_it) {  // past the end, or a row that no sequence owns
          if (!direct || q.t0 + i < a.T) {
            store(static_cast<IO*>(a.out), elem(q, 0, i), i, both(0.f), direct);
            if (kDown) store(static_cast<IO*>(a.dg), second(i), i, both(0.f), direct);
          }
          continue;
        }
        if constexpr (!kDown) {
          h = starts ? in[r] : fma2(al[r], h, in[r]);
          store(static_cast<IO*>(a.out), elem(q, 0, i), i, in_it ? h : both(0.f), direct);
        } else {
          f2 z, x = load2(q, 0, i);
          if constexpr (kFrom) z = codes_of(q, 2, i);
          else {
            if (E == 2 && stops) z = state_of(q, a.h0, row_info(q, i).seq);
            else z = load2(q, 2, i);
            if (E == 1) z = stops ? ends : z;
            if (COMPL) z = add2(z, neg2(load2(q, 3, i)));
          }
          f2 from = h;
          if (E == 1) from = starts ? begins : h, x = in_it ? x : both(0.f);
          if (E == 2 && starts) from = state_of(q, a.s0, row_info(q, i).seq);
          const f2 d = add2(x, from);
          h = mul2(al[r], d);
          f2 dg = mul2(h, z);
          if (RAW) dg = mul2(dg, in[r]);
          const f2 dx = COMPL ? mul2(in[r], d) : d;
          store(static_cast<IO*>(a.out), elem(q, 0, i), i, in_it ? dx : both(0.f), direct);
          store(static_cast<IO*>(a.dg), second(i), i, in_it ? dg : both(0.f), direct);
        }
        if (E == 1) final = stops ? h : final;
        if (E == 2 && stops && a.sT) state_out(h, i);
      }
      if (E == 1 && stop && a.sT) state_out(final, row_at(__ffs(stop) - 1));
    };
    if (kind == 1) {
      emit(integral_constant<int, 1>{}, std::true_type{});
    } else if (kind == 2) {
      emit(integral_constant<int, 2>{}, std::true_type{});
    } else if (p.tma) {
      emit(integral_constant<int, 0>{}, std::true_type{});
    } else {
      emit(integral_constant<int, 0>{}, std::false_type{});
    }

    // ---- out by TMA, each unit's rows (rows past T are not written)
    if (p.tma) {
      fence_async_smem();
      __syncwarp();
      if (lane == 0 && q.t0 + lowest < a.T) {
        const int at = lowest * W * (int)sizeof(IO), t = q.t0 + lowest;
        tma_store_3d(&p.out[0], q.st + at, q.cb * W, t, q.b);
        if (kDown) tma_store_3d(&p.out[1], (kFrom ? stages + NS * S::kStage : q.st + S::at(1)) + at, q.cb * W, t, q.b);
        bulk_commit();
      }
    }
  }
  if (sh.lost[(k + 1) & 1]) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (threadIdx.x == 0)  // its copies in flight
      for (int j = k - 1; j < k + 2; ++j) wait_for(&sh.full[j % NS], (j / NS) & 1);
  }
  if (lane == 0) bulk_wait_read();
  __syncwarp();
  // a block's shared memory stays until the others have sent what they send
  if (size > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr float kLeast = -128.f;  // lambda in the checkpoint: exp is zero in fp32 from there on

// log(1 + e) for 0 <= e <= 1, as 2 artanh(s) with s = e / (2 + e) <= 1/3 (the series to s^13, 3e-8 off).
__device__ __forceinline__ f2 log1p2_of(f2 e) {
  float a, b;
  unpack(add2(e, both(2.f)), a, b);
  const f2 s = mul2(e, pack(rcp_of(a), rcp_of(b))), q = mul2(s, s);
  f2 t = fma2(q, both(2.f / 13.f), both(2.f / 11.f));
  t = fma2(q, t, both(2.f / 9.f));
  t = fma2(q, t, both(2.f / 7.f));
  t = fma2(q, t, both(2.f / 5.f));
  t = fma2(q, t, both(2.f / 3.f));
  t = fma2(q, t, both(2.f));
  return mul2(s, t);
}

// The 8-bit checkpoint.  A block writes 128 channels (a row's scale block) of
// four segments of the forward's rows; a thread holds two channels x one
// segment, as there, and goes the same way from the state that entered the
// segment, so that z is what the forward saw.  In bf16 it touches 6.3 B per
// element: x and g once more (from L2 for the rows that the forward did last,
// which come first here), the two codes, the states; 5.5 of them in DRAM (33.5 M
// elements, 96 us).  58 instructions an element, issued on 60 % of the cycles.
// All loads of a thread are in flight at once.
template <typename IO, bool RAW, bool COMPL>
__global__ void __launch_bounds__(256, 2) scan_save_kernel(const __grid_constant__ TileArgs p) {
  using S = Shape<kFwd, IO, COMPL>;
  constexpr int R = S::kR, kSegs = 4;
  __shared__ uint32_t top[8][2][R];  // of a warp's rows, lambda and z: the largest magnitude
  __shared__ float inv[kSegs][2][R];
  const ScanArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, across = threadIdx.x % 64, seg = threadIdx.x / 64;
  const int kb = (a.D + kBlock - 1) / kBlock, parts = (a.T + kSegs * R - 1) / (kSegs * R);
  const int cb = blockIdx.x % kb, b = blockIdx.x / kb % a.B, part = parts - 1 - (int)(blockIdx.x / kb / a.B);
  const int c = cb * kBlock + across * 2, n = a.D - c;
  const int t0 = (part * kSegs + seg) * R, most = min(R, a.T - t0);  // rows of this thread: the first `most` exist
  const size_t rows = (size_t)a.B * a.T, row0 = (size_t)b * a.T + t0;
  const ScanCkptLayout lay = scan_ckpt_layout(rows, a.D);
  // the rows as loaded, two channels in a word (bf16) or two
  constexpr int kWords = sizeof(IO) / 2;
  uint32_t x[R][kWords], g[R][kWords];
  const bool pairs = a.D % 2 == 0;
  const IO *px = static_cast<const IO*>(a.x) + row0 * a.D + c, *pg = static_cast<const IO*>(a.g) + row0 * a.D + c;
  if (pairs && n > 0 && most == R) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        x[r][j] = __ldg(reinterpret_cast<const uint32_t*>(px + (size_t)r * a.D) + j);
        g[r][j] = __ldg(reinterpret_cast<const uint32_t*>(pg + (size_t)r * a.D) + j);
      }
  } else {
    auto load = [&](const IO* q, bool in, uint32_t* to) {
      IO v[2] = {in && n > 0 ? q[0] : from_f32<IO>(0.f), in && n > 1 ? q[1] : from_f32<IO>(0.f)};
#pragma unroll
      for (int j = 0; j < kWords; ++j) to[j] = reinterpret_cast<const uint32_t*>(v)[j];
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
      load(px + (size_t)r * a.D, r < most, x[r]);
      load(pg + (size_t)r * a.D, r < most, g[r]);
    }
  }
  auto value = [](const uint32_t* w) {
    if constexpr (kWords == 1)
      return pack(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u));
    else
      return pack(__uint_as_float(w[0]), __uint_as_float(w[1]));
  };
  grid_dep_wait();  // what entered the segments comes from the kernel before
  // bit r: whether row r belongs to a sequence, and whether it is one's first
  uint32_t valid = most > 0 ? (1u << most) - 1 : 0, first = t0 == 0 ? 1 : 0;
  if (a.cu) {
    valid = first = 0;
    for (int r = 0; r < most; ++r) {
      const int v = __ldg(p.info + t0 + r);
      valid |= (v >= 0 ? 1u : 0u) << r, first |= (v >= 0 && (v & 2) ? 1u : 0u) << r;
    }
  }
  auto state_of = [&](int r) {
    float v[2];
    const int seq = a.cu ? __ldg(p.info + t0 + r) >> 2 : b;
    ldg<2>(a.s0 ? a.s0 + (size_t)seq * a.D + c : nullptr, v, n, pairs);
    return pack(v[0], v[1]);
  };
  f2 h = both(0.f), z[R], lam[R];
  if (n > 0 && most > 0) {
    const size_t chain = (size_t)b * p.blocks + c / S::W, segs = (size_t)p.chunks * kWarps * S::kSide;
    const float2 e = *reinterpret_cast<const float2*>(p.enters + (chain * segs + part * kSegs + seg) * S::W + c % S::W);
    h = pack(e.x, e.y);
  }
  auto rows_of = [&](auto edges) {
    constexpr bool E = decltype(edges)::value;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const f2 gv = value(g[r]);
      f2 al, be = 0;
      gate<RAW, COMPL>(gv, al, be);
      if (E && (first >> r & 1)) h = state_of(r);
      z[r] = COMPL ? add2(h, neg2(value(x[r]))) : h;
      const f2 u = COMPL ? mul2(be, value(x[r])) : value(x[r]);
      if (!E || (valid >> r & 1)) h = fma2(al, h, u);
      float f[2];
      unpack(gv, f[0], f[1]);
      lam[r] = pack(max_nan(f[0], kLeast), max_nan(f[1], kLeast));
      if (RAW) {  // min(g, 0) - log(1 + exp(-|g|))
        const f2 l = log1p2_of(exp2_of(pack(-min_nan(fabsf(f[0]), 128.f), -min_nan(fabsf(f[1]), 128.f))));
        lam[r] = add2(pack(max_nan(min_nan(f[0], 0.f), kLeast), max_nan(min_nan(f[1], 0.f), kLeast)), neg2(l));
      }
      if (E) {
        const bool in = valid >> r & 1;
        unpack(lam[r], f[0], f[1]);
        lam[r] = pack(in && n > 0 ? f[0] : 0.f, in && n > 1 ? f[1] : 0.f);
        unpack(z[r], f[0], f[1]);
        z[r] = pack(in && n > 0 ? f[0] : 0.f, in && n > 1 ? f[1] : 0.f);
      }
    }
  };
  if (first || valid != (1u << R) - 1 || n < 2)
    rows_of(std::true_type{});
  else
    rows_of(std::false_type{});
  // the largest magnitudes; non-finite values, which do not count, are looked for only where there are any
  auto tops = [&](auto careful) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float f[2];
        unpack(m ? z[r] : lam[r], f[0], f[1]);
        const uint32_t u0 = decltype(careful)::value ? magnitude(f[0]) : __float_as_uint(f[0]) & 0x7fffffffu;
        const uint32_t u1 = decltype(careful)::value ? magnitude(f[1]) : __float_as_uint(f[1]) & 0x7fffffffu;
        const uint32_t t = __reduce_max_sync(0xffffffffu, max(u0, u1));
        if (lane == 0) top[warp][m][r] = t;
      }
    __syncthreads();
    bool odd = false;
    if (across < 2 * R) {  // one scale each
      const int m = across / R, r = across % R;
      const uint32_t t = max(top[2 * seg][m][r], top[2 * seg + 1][m][r]);
      odd = t >= 0x7f800000u;
      const int code = scale_code(__uint_as_float(t));
      inv[seg][m][r] = pow2(254 - code);
      if (r < most && !odd) a.ckpt[(m ? lay.z_scale : lay.lam_scale) + cb * rows + row0 + r] = (uint8_t)code;
    }
    return __syncthreads_or(odd);
  };
  auto codes = [&](auto careful) {
    if (n <= 0) return;
    uint8_t* to = a.ckpt + row0 * lay.pitch + c;
#pragma unroll
    for (int r = 0; r < R; ++r, to += lay.pitch) {
      if (r >= most) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float f[2];
        const float by = inv[seg][m][r];
        if (decltype(careful)::value) {
          unpack(m ? z[r] : lam[r], f[0], f[1]);
          f[0] = finite(f[0]) ? f[0] * by : __int_as_float(0x7fffffff);
          f[1] = finite(f[1]) ? f[1] * by : __int_as_float(0x7fffffff);
        } else {
          unpack(mul2(m ? z[r] : lam[r], both(by)), f[0], f[1]);
        }
        *reinterpret_cast<uint16_t*>(to + (m ? lay.z : 0)) =
            __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
      }
    }
  };
  if (tops(std::false_type{})) {
    tops(std::true_type{});
    codes(std::true_type{});
  } else {
    codes(std::false_type{});
  }
}

// Before a sequence call: header and ticket cleared, the words that blocks
// hand to each other marked as not written; packed: what each row is, and the
// states of the empty sequences, whose final state is their initial state.
__global__ void __launch_bounds__(256) scan_init_kernel(const TileArgs p, uint4* words, size_t count, int32_t* info) {
  grid_dep_launch();
  grid_dep_wait();
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x, step = (size_t)gridDim.x * 256;
  if (at < sizeof(WorkspaceHeader) / 4) reinterpret_cast<uint32_t*>(p.hdr)[at] = 0;
  for (size_t i = at; i < count; i += step) words[i] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
  const ScanArgs& a = p.a;
  if (!a.cu) return;
  const size_t padded = (size_t)a.T + kInfoPad;  // tiles are read whole
  for (size_t t = at; t < padded; t += step) {
    if (t >= (size_t)a.T) {
      info[t] = -1;
      continue;
    }
    int lo = 0, hi = a.N + 1;  // the first of cu[0 .. N] that is past t
    while (lo < hi) {
      const int m = lo + (hi - lo) / 2;
      if ((int64_t)__ldg(a.cu + m) <= (int64_t)t)
        lo = m + 1;
      else
        hi = m;
    }
    int v = -1;
    if (lo > 0 && lo <= a.N)
      v = (lo - 1) * 4 + ((size_t)__ldg(a.cu + lo - 1) == t ? 2 : 0) + ((int64_t)__ldg(a.cu + lo) - 1 == (int64_t)t ? 1 : 0);
    info[t] = v;
  }
  if (!a.sT || a.sT == a.s0) return;
  for (int i = blockIdx.x; i < a.N; i += gridDim.x)
    if (__ldg(a.cu + i + 1) <= __ldg(a.cu + i))
      for (int c = threadIdx.x; c < a.D; c += 256) a.sT[(size_t)i * a.D + c] = a.s0 ? a.s0[(size_t)i * a.D + c] : 0.f;
}

// One token: a stream over state, x, g and h (14 B per element in bf16); four
// channels per thread.
template <typename IO, bool RAW, bool COMPL>
__global__ void __launch_bounds__(256) scan_step_kernel(const IO* __restrict__ x, const IO* __restrict__ g,
                                                        const float* state, float* out_state, IO* __restrict__ h,
                                                        size_t count) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  const int n = (int)min((size_t)4, count - i);
  float gv[4], xv[4], s[4];
  if (n == 4) {
    lds<IO, 4>(reinterpret_cast<const uint8_t*>(g + i), gv);
    lds<IO, 4>(reinterpret_cast<const uint8_t*>(x + i), xv);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) gv[j] = j < n ? to_f32(g[i + j]) : 0.f, xv[j] = j < n ? to_f32(x[i + j]) : 0.f;
  }
  ldg<4>(state + i, s, n, n == 4);
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    f2 alpha, beta = 0;
    gate<RAW, COMPL>(pack(gv[j], gv[j + 1]), alpha, beta);
    const f2 v = pack(xv[j], xv[j + 1]);
    unpack(fma2(alpha, pack(s[j], s[j + 1]), COMPL ? mul2(beta, v) : v), s[j], s[j + 1]);
  }
  stg<4>(out_state + i, s, n, n == 4);
  stg<4>(h + i, s, n, n == 4);
}

// ========================================================================= host
// Calls f with the flags as compile-time constants.
template <typename F>
cudaError_t with_flags(int dtype, int prep, int complement, F f) {
  using std::false_type;
  using std::true_type;
  const bool raw = prep & KDA_PREP_GATE_LOGSIGMOID;
  auto inner = [&](auto io) {
    if (raw) return complement ? f(io, true_type{}, true_type{}) : f(io, true_type{}, false_type{});
    return complement ? f(io, false_type{}, true_type{}) : f(io, false_type{}, false_type{});
  };
  return dtype == KDA_F32 ? inner(float{}) : inner(__nv_bfloat16{});
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// [B][T][row of `pitch` elements, `width` of them read]; box: a tile.
bool make_map(CUtensorMap* map, const void* base, int eb, int B, int T, size_t width, size_t pitch, int box_width,
              int box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  const CUtensorMapDataType type = eb == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : eb == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  cuuint64_t dims[3] = {width, (cuuint64_t)T, (cuuint64_t)B};
  cuuint64_t strides[2] = {pitch * eb, pitch * eb * (cuuint64_t)T};
  cuuint32_t box[3] = {(cuuint32_t)box_width, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
  return enc(map, type, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
size_t info_bytes(int T) { return align256(((size_t)T + kInfoPad) * 4); }

constexpr int kSms = 148;  // of a B200; a launch is sized for it, results do not depend on it

// How a call of these sizes goes: the blocks that walk a chain together (0:
// kJoin), and what it keeps in the workspace.
struct Plan {
  int64_t chains, chunks, groups;
  int cluster;
  size_t pair_words, state_words;  // to be marked as not written
};
Plan plan_of(int64_t B, int64_t T, int64_t D, int width, int rows, int per_sm) {
  Plan q{};
  q.chains = B * div_up(D, width), q.chunks = div_up(T, rows);
  if (q.chains < kJoinChains && q.chunks > kJoinTiles) {
    q.groups = div_up(q.chunks, kGroup);
    q.pair_words = (size_t)(q.chains * q.chunks * 2 * width);
    q.state_words = (size_t)(q.chains * q.groups * width);
  } else {
    q.cluster = 1;
    while (q.cluster < kCluster && q.chains * q.cluster * 2 <= kSms * per_sm && q.cluster * 2 <= q.chunks) q.cluster *= 2;
  }
  return q;
}
template <Kind K, typename IO, bool COMPL>
Plan plan_for(int64_t B, int64_t T, int64_t D) {
  using S = Shape<K, IO, COMPL>;
  return plan_of(B, T, D, S::W, S::kL, S::kPerSm);
}

// `after`: the kernel waits for the one before it by itself; cluster: of so many blocks.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, bool after,
                   int cluster, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  if (after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster, attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <Kind K, typename IO, bool RAW, bool COMPL>
cudaError_t launch_tiles(const ScanArgs& a, void* ws, cudaStream_t stream) {
  using S = Shape<K, IO, COMPL>;
  TileArgs p;
  p.a = a;
  const Plan plan = plan_for<K, IO, COMPL>(a.B, a.T, a.D);
  p.blocks = (int)div_up(a.D, S::W);
  p.chains = (int)plan.chains, p.chunks = (int)plan.chunks, p.groups = (int)plan.groups;
  p.cluster = plan.cluster;
  p.vec = a.D % 4 == 0;
  p.tma = (size_t)a.D * sizeof(IO) % 16 == 0;
  p.words = (size_t)a.D * sizeof(IO) % 4 == 0;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.hdr = reinterpret_cast<WorkspaceHeader*>(w);
  w += sizeof(WorkspaceHeader);
  p.pairs = reinterpret_cast<float*>(w);
  p.states = p.pairs + plan.pair_words;
  w += align256((plan.pair_words + plan.state_words) * 4);
  int32_t* info = reinterpret_cast<int32_t*>(w);
  p.info = info;
  if (a.cu) w += info_bytes(a.T);
  p.enters = K == kFwd && a.ckpt ? reinterpret_cast<float*>(w) : nullptr;
  const void* arrays[4] = {a.x, a.g, nullptr, nullptr};
  if (S::kDown) arrays[0] = a.dy, arrays[1] = a.g, arrays[2] = a.h, arrays[3] = a.x;
  const ScanCkptLayout l = scan_ckpt_layout((size_t)a.B * a.T, a.D);
  bool ok = true;
  for (int i = 0; i < S::kIn; ++i) {
    if (S::kFrom && i > 0)
      ok = ok && make_map(&p.map[i], a.ckpt + (i == 2 ? l.z : 0), 1, a.B, a.T, a.D, l.pitch, S::W, S::kL);
    else if (p.tma)
      ok = ok && make_map(&p.map[i], arrays[i], sizeof(IO), a.B, a.T, a.D, a.D, S::W, S::kL);
  }
  if (p.tma) ok = ok && make_map(&p.out[0], a.out, sizeof(IO), a.B, a.T, a.D, a.D, S::W, S::kUnitRows);
  if (p.tma && S::kDown) ok = ok && make_map(&p.out[1], a.dg, sizeof(IO), a.B, a.T, a.D, a.D, S::W, S::kUnitRows);
  if (!ok) return cudaErrorInvalidValue;
  auto kernel = scan_tile_kernel<K, IO, RAW, COMPL>;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit has been raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit) || !bit) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const bool init = !p.cluster || a.cu;
  if (init) {
    const size_t count = (plan.pair_words + plan.state_words) / 4;
    const int64_t blocks = std::max(div_up((int64_t)count, 256 * 4), div_up(a.cu ? a.T + kInfoPad : 1, 256));
    e = launch(scan_init_kernel, (unsigned)std::min<int64_t>(blocks, kSms * 8), 256, 0, stream, false, 1, p,
               reinterpret_cast<uint4*>(p.pairs), count, info);
    if (e != cudaSuccess) return e;
  }
  const int64_t grid = p.cluster ? plan.chains * p.cluster : std::min<int64_t>(plan.chains * plan.chunks, kSms * S::kPerSm);
  // Clusters are not launched before the kernel ahead has left: started beside its blocks they come to lie unevenly
  // on the SMs and stay so (166 us against 98 for 32767 packed rows of 1024 channels).
  e = launch(kernel, (unsigned)grid, kThreads, S::kSmem, stream, init && !p.cluster, p.cluster, p);
  if constexpr (K == kFwd) {
    if (e == cudaSuccess && a.ckpt)
      e = launch(scan_save_kernel<IO, RAW, COMPL>,
                 (unsigned)(div_up(a.D, kBlock) * a.B * div_up(a.T, 4 * S::kR)), 256, 0, stream, true, 1, p);
  }
  return e;
}

}  // namespace

// Enough for every kind of call of these sizes: the header, whose error word
// tells of a wait that gave up, the words handed between blocks, the rows'
// information if packed, the forward's states at its segments for the
// checkpoint.
size_t scan_workspace_bytes(int B, int T, int D, int N, int dtype, bool checkpoint) {
  if (B == 0 || T == 0) return 0;
  size_t words = 0, enters = 0;
  const auto fit = [&](const Plan& q) { words = std::max(words, q.pair_words + q.state_words); };
  const auto fit_all = [&](auto io) {
    using IO = decltype(io);
    const Plan f = plan_for<kFwd, IO, false>(B, T, D);
    enters = (size_t)(f.chains * f.chunks) * kWarps * Shape<kFwd, IO, false>::kSide * Shape<kFwd, IO, false>::W;
    fit(f), fit(plan_for<kFwd, IO, true>(B, T, D));
    fit(plan_for<kBwd, IO, false>(B, T, D)), fit(plan_for<kBwd, IO, true>(B, T, D));
    fit(plan_for<kBwdCkpt, IO, false>(B, T, D)), fit(plan_for<kBwdCkptNarrow, IO, false>(B, T, D));
  };
  if (dtype == KDA_F32)
    fit_all(float{});
  else
    fit_all(__nv_bfloat16{});
  return sizeof(WorkspaceHeader) + align256(words * 4) + (N > 0 ? info_bytes(T) : 0) +
         (checkpoint ? align256(enters * 4) : 0);
}

cudaError_t launch_scan_fwd(const ScanArgs& a, void* ws, cudaStream_t stream) {
  return with_flags(a.dtype, a.prep, a.complement, [&](auto io, auto raw, auto compl_) {
    return launch_tiles<kFwd, decltype(io), raw.value, compl_.value>(a, ws, stream);
  });
}

cudaError_t launch_scan_bwd(const ScanArgs& a, void* ws, cudaStream_t stream) {
  return with_flags(a.dtype, a.prep, a.complement, [&](auto io, auto raw, auto compl_) {
    using IO = decltype(io);
    if (!a.ckpt) return launch_tiles<kBwd, IO, raw.value, compl_.value>(a, ws, stream);
    if constexpr (sizeof(IO) == 2)
      if ((int64_t)a.B * div_up(a.D, 64) >= kWideChains)
        return launch_tiles<kBwdCkpt, IO, raw.value, compl_.value>(a, ws, stream);
    return launch_tiles<kBwdCkptNarrow, IO, raw.value, compl_.value>(a, ws, stream);
  });
}

cudaError_t launch_scan_step(const void* x, const void* g, const float* state, float* out_state, void* h, size_t n,
                             int dtype, int prep, int complement, cudaStream_t stream) {
  return with_flags(dtype, prep, complement, [&](auto io, auto raw, auto compl_) {
    using IO = decltype(io);
    scan_step_kernel<IO, raw.value, compl_.value><<<(unsigned)((n + 1023) / 1024), 256, 0, stream>>>(
        static_cast<const IO*>(x), static_cast<const IO*>(g), state, out_state, static_cast<IO*>(h), n);
    return cudaGetLastError();
  });
}

}  // namespace kda
