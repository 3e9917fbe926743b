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
// the 8-bit checkpoint 8.  So the data is read once, in one pass: a tile is
// 128 channels (one scale block of the checkpoint) x L rows; each of 8 warps
// holds R = L / 8 rows x 128 channels of a tile as alpha and input in
// registers and folds them to (A, Bs).  Then one thread per channel folds the
// 8 pairs and walks the state through them, so that each warp finds what
// enters its rows and goes over them once more.  Tiles of one (batch, channel
// block) chain are joined in the order of the rows: each tile publishes its
// (A, Bs), the last of each group of kGroup tiles the state that leaves the
// group; a tile folds the pairs of its group's earlier tiles onto the state
// that left the group before.  The order of the fold is fixed, so the bits are
// the same every time.  Tiles are drawn by ticket in the order of the rows, so
// whatever a tile waits for belongs to a block that is running; the words of
// the pairs are their own flags (all bits set = not yet written), so one trip
// to L2 sees and fetches them.  While four warps do this, another draws the
// next ticket and starts the tile after next on its way (TMA, three stages).
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
constexpr int kBlock = 128;     // channels per tile and per scale of the checkpoint
constexpr int kWarps = 8;
constexpr int kFeeder = 7;      // the warp that draws tickets and starts loads
constexpr int kGroup = 16;      // tiles whose pairs are folded before a state is published
constexpr int kStages = 3;
constexpr int kInOrderRows = 256;  // chains of so few rows are walked by one block each
constexpr uint32_t kEmpty = 0xffffffffu;     // a word not yet written
constexpr uint32_t kPollLimit = 1u << 22;    // polls before a wait gives up
constexpr uint32_t kBarLimit = 1u << 22;

// exp(x) for x <= 126 ln 2, to about two ulp: 2^p for p = x / ln 2 rounded,
// times 1 + (x - p ln 2), what the rounding left out.  x = -infinity gives NaN.
__device__ __forceinline__ float exp_of(float x) {
  const float p = x * 1.44269504f;
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(p));
  return fmaf(e, fmaf(p, -0.693147181f, x), e);
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
// 1 - exp(x) for x <= 0 given alpha = exp(x): the series where the difference
// would lose the small rates that make the long memories.
__device__ __forceinline__ float rate_of(float x, float alpha) {
  float q = fmaf(x, 1.f / 40320.f, 1.f / 5040.f);
  q = fmaf(x, q, 1.f / 720.f);
  q = fmaf(x, q, 1.f / 120.f);
  q = fmaf(x, q, 1.f / 24.f);
  q = fmaf(x, q, 1.f / 6.f);
  q = fmaf(x, q, 0.5f);
  q = fmaf(x, q, 1.f);
  return fabsf(x) < 0.5f ? -x * q : 1.f - alpha;
}
// alpha and 1 - alpha of a gate, each to a few ulp on its own.  The clamps
// keep the exponent's residual a number; past them exp is below 2^-126 and
// counts as zero.  NaN stays NaN.
template <bool RAW>
__device__ __forceinline__ void gate(float g, float& alpha, float& beta) {
  if (RAW) {
    const float e = exp_of(-min_nan(fabsf(g), 128.f)), hi = rcp_of(1.f + e), lo = e * hi;
    alpha = g >= 0.f ? hi : lo;
    beta = g >= 0.f ? lo : hi;
  } else {
    const float x = max_nan(g, -128.f);
    alpha = exp_of(x);
    beta = rate_of(x, alpha);
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
// Four values as e4m3 of v * inv (inv a power of two; non-finite values give NaN).
__device__ __forceinline__ uint32_t encode4(const float* v, float inv) {
  float q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = finite(v[j]) ? v[j] * inv : __int_as_float(0x7fffffff);
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ void decode4(uint32_t c, float scale, float* v) {
  const __half2 a = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3));
  const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3));
  const float2 x = __half22float2(a), y = __half22float2(b);
  v[0] = x.x * scale, v[1] = x.y * scale, v[2] = y.x * scale, v[3] = y.y * scale;
}


// ------------------------------------------------------------ four channels
template <typename IO>
__device__ __forceinline__ void lds4(const uint8_t* p, float* v) {
  if constexpr (sizeof(IO) == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
  }
}
template <typename IO>
__device__ __forceinline__ void stg4(IO* p, const float* v, int n, bool vec) {
  if (vec) {
    if (n <= 0) return;
    if constexpr (sizeof(IO) == 4) {
      __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      __stcs(reinterpret_cast<uint2*>(p),
             make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = from_f32<IO>(v[j]);
  }
}
__device__ __forceinline__ void ldg4(const float* p, float* v, int n, bool vec) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = 0.f;
  if (!p || n <= 0) return;
  if (vec) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) v[j] = p[j];
  }
}

// ------------------------------------------------------------- pairs (A, Bs)
__device__ __forceinline__ bool fresh(float A) { return __float_as_uint(A) == 0x80000000u; }
// What leaves a stretch (A, B) that c enters.
__device__ __forceinline__ float through(float c, float A, float B) { return fresh(A) ? B : fmaf(A, c, B); }

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
enum Kind { kFwd, kFwdCkpt, kBwd, kBwdCkpt };

// Input arrays of a stage, and rows per warp: a stage is 24 or 32 KiB, three
// of them and two blocks per SM (the fp32 backward: 48 or 64 KiB, one block).
template <Kind K, typename IO, bool COMPL>
struct Shape {
  static constexpr bool kDown = K == kBwd || K == kBwdCkpt;
  static constexpr int kIn = K == kBwd ? (COMPL ? 4 : 3) : K == kBwdCkpt ? 3 : 2;
  static constexpr int kRows = sizeof(IO) == 4 || K == kBwd ? 4 : 8;  // per warp
  static constexpr int kL = kWarps * kRows;
  // element bytes of array i: forward x, g; backward dy, g, h, x; from the checkpoint dy, lambda, z
  __host__ __device__ static constexpr int eb(int i) { return K == kBwdCkpt && i > 0 ? 1 : (int)sizeof(IO); }
  __host__ __device__ static constexpr int at(int i) {
    int o = 0;
    for (int j = 0; j < i; ++j) o += kL * kBlock * eb(j);
    return o;
  }
  static constexpr int kStage = at(kIn);
  static constexpr int kSmem = kStages * kStage;
  static constexpr int kPerSm = kSmem > 96 * 1024 ? 1 : 2;
};

struct TileArgs {
  ScanArgs a;
  CUtensorMap map[4];
  WorkspaceHeader* hdr;     // error word; pad[0] is the ticket
  float* pairs;             // [chains][chunks][2][128]
  float* states;            // [chains][groups][128]
  const int32_t* info;      // packed: sequence * 4 + first * 2 + last of each row, -1 outside
  int chains, chunks, groups, blocks;  // blocks: of channels
  bool tma, vec, in_order;
};

struct __align__(16) Shared {
  float pair[kWarps][2][kBlock];  // (A, Bs) of each warp's rows
  float enter[kWarps][kBlock];    // what enters them
  float carry[kBlock];            // in order: what leaves the tile
  uint64_t full[kStages];
  int tile[kStages];
  int info[kStages][64];
  uint8_t scale[kStages][2][64];
};

struct Row {
  bool valid, first, last;
  int seq;
};

template <Kind K, typename IO, bool RAW, bool COMPL>
__global__ void __launch_bounds__(32 * kWarps, Shape<K, IO, COMPL>::kPerSm)
    scan_tile_kernel(const __grid_constant__ TileArgs p) {
  using S = Shape<K, IO, COMPL>;
  constexpr int R = S::kRows, L = S::kL;
  constexpr bool kDown = S::kDown, kSave = K == kFwdCkpt, kFrom = K == kBwdCkpt;
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ Shared sh;
  const ScanArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t rows = (size_t)a.B * a.T;
  const bool packed = a.cu != nullptr;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sh.full[s], 2);
    fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();  // the workspace was prepared, and the inputs written, by earlier kernels

  auto gave_up = [&](uint32_t where) {
    if (!p.hdr) return;
    atomicOr(&p.hdr->error, 1u);
    atomicExch(&p.hdr->where, where);
  };
  auto first_row = [&](int chunk) { return (kDown ? p.chunks - 1 - chunk : chunk) * (int64_t)L; };

  // ---- the feeder: tile `it` of this block into its stage
  uint32_t drawn = 0;  // lane 0: the next ticket
  if (warp == kFeeder && lane == 0 && !p.in_order) drawn = atomicAdd(&p.hdr->pad[0], 1u);
  bool fed_all = false;
  auto feed = [&](int it) {
    if (fed_all) return;
    const int s = it % kStages;
    int tile;
    if (p.in_order) {
      tile = it < p.chunks ? it * p.chains + (int)blockIdx.x : -1;
    } else {
      const uint32_t t = __shfl_sync(0xffffffffu, drawn, 0);
      tile = t < (uint32_t)p.chains * (uint32_t)p.chunks ? (int)t : -1;
      if (tile >= 0 && lane == 0) drawn = atomicAdd(&p.hdr->pad[0], 1u);
    }
    if (lane == 0) sh.tile[s] = tile;
    if (tile < 0) {
      if (lane == 0) mbar_arrive(&sh.full[s]), mbar_arrive(&sh.full[s]);
      fed_all = true;
      return;
    }
    const int chain = tile % p.chains, chunk = tile / p.chains, b = chain / p.blocks, cb = chain % p.blocks;
    const int64_t t0 = first_row(chunk);
    if (lane == 0 && p.tma) {
      mbar_expect_tx(&sh.full[s], S::kStage);
#pragma unroll
      for (int i = 0; i < S::kIn; ++i)  // h one row up: what enters each row
        tma_load_3d(stages + s * S::kStage + S::at(i), &p.map[i], &sh.full[s], cb * kBlock,
                    (int)t0 - (K == kBwd && i == 2 ? 1 : 0), b);
    }
    if (packed)
      for (int i = lane; i < L; i += 32) sh.info[s][i] = t0 + i < a.T ? p.info[t0 + i] : -1;
    if (kFrom) {
      const ScanCkptLayout l = scan_ckpt_layout(rows, a.D);
      for (int i = lane; i < L; i += 32) {
        const size_t at = cb * rows + (size_t)b * a.T + t0 + i;
        sh.scale[s][0][i] = t0 + i < a.T ? a.ckpt[l.lam_scale + at] : 1;
        sh.scale[s][1][i] = t0 + i < a.T ? a.ckpt[l.z_scale + at] : 1;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.full[s]);
    if (lane == 0 && !p.tma) mbar_arrive(&sh.full[s]);
  };
  if (warp == kFeeder) feed(0), feed(1);

  bool failed = false;
  for (int it = 0;; ++it) {
    const int s = it % kStages;
    const bool there = mbar_wait(&sh.full[s], (it / kStages) & 1, kBarLimit);
    if (!there) gave_up(202);
    const int tile = there ? sh.tile[s] : -1;
    if (tile < 0) break;
    const int chain = tile % p.chains, chunk = tile / p.chains, b = chain / p.blocks, cb = chain % p.blocks;
    const int64_t t0 = first_row(chunk);
    const int c = cb * kBlock + lane * 4, n = a.D - c;  // this lane's channels, and how many there are (from 4 up: 4)
    uint8_t* st = stages + s * S::kStage;
    // row i of the tile that this warp handles r-th
    auto row_at = [&](int r) { return kDown ? L - 1 - (warp * R + r) : warp * R + r; };
    auto elem = [&](int arr, int i) { return st + S::at(arr) + (i * kBlock + lane * 4) * S::eb(arr); };
    auto global_row = [&](int i) { return (size_t)b * a.T + t0 + i; };

    if (!p.tma) {
      // rows that TMA cannot take: each lane brings its own four channels
      for (int r = 0; r < R; ++r) {
        const int i = row_at(r);
        const bool in = t0 + i < a.T;
#pragma unroll
        for (int arr = 0; arr < S::kIn; ++arr) {
          if (kFrom && arr > 0) {
            const ScanCkptLayout l = scan_ckpt_layout(rows, a.D);
            uint32_t v = 0;
            if (in && n > 0)
              v = *reinterpret_cast<const uint32_t*>(a.ckpt + (arr == 2 ? l.z : 0) + global_row(i) * l.pitch + c);
            *reinterpret_cast<uint32_t*>(elem(arr, i)) = v;
            continue;
          }
          const void* src = K == kFwd || K == kFwdCkpt ? (arr == 0 ? a.x : a.g)
                                                       : (arr == 0 ? a.dy : arr == 1 ? a.g : arr == 2 ? a.h : a.x);
          const bool up = K == kBwd && arr == 2;
          const bool ok = in && (!up || t0 + i > 0);
          const IO* q = static_cast<const IO*>(src) + (ok ? (global_row(i) - up) * a.D + c : 0);
          IO* d = reinterpret_cast<IO*>(elem(arr, i));
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = ok && j < n ? q[j] : from_f32<IO>(0.f);
        }
      }
      __syncwarp();
    }

    auto row_info = [&](int i) {
      Row q;
      if (packed) {
        const int v = sh.info[s][i];
        q.valid = v >= 0, q.first = v & 2, q.last = v & 1, q.seq = v >> 2;
      } else {
        const int64_t t = t0 + i;
        q.valid = t < a.T, q.first = t == 0, q.last = t == a.T - 1, q.seq = b;
      }
      return q;
    };
    // whether any of the warp's rows starts or ends a sequence or belongs to none
    bool edge = false;
    if (lane < R) {
      const Row q = row_info(row_at(lane));
      edge = !q.valid || q.first || q.last;
    }
    edge = __any_sync(0xffffffffu, edge);
    auto state_of = [&](const float* base, int seq, float* v) {
      ldg4(base ? base + (size_t)seq * a.D + c : nullptr, v, n, p.vec);
    };
    auto load_gate = [&](int i, float* g) {
      if constexpr (kFrom)
        decode4(*reinterpret_cast<const uint32_t*>(elem(1, i)), pow2(sh.scale[s][0][i]), g);
      else
        lds4<IO>(elem(1, i), g);
    };

    // ---- the warp's rows as one pair
    float al[R][4], u[R][4];  // alpha; forward: the input, backward: 1 - alpha
    float A[4], B[4];
    auto reduce = [&](auto edges) {
#pragma unroll
      for (int j = 0; j < 4; ++j) A[j] = 1.f, B[j] = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = row_at(r);
        float g[4], v[4];
        load_gate(i, g);
        lds4<IO>(elem(0, i), v);
        const Row q = edges.value ? row_info(i) : Row{true, false, false, 0};
        float from[4];
        const bool start = edges.value && q.valid && (kDown ? q.last : q.first);
        if (start) state_of(a.s0, q.seq, from);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float be;
          gate<RAW && !kFrom>(g[j], al[r][j], be);
          u[r][j] = kDown ? be : COMPL ? be * v[j] : v[j];
          if (edges.value && !q.valid) continue;
          if (start) {
            if (!kDown) u[r][j] = fmaf(al[r][j], from[j], u[r][j]);
            A[j] = -0.f;
            B[j] = kDown ? al[r][j] * (v[j] + from[j]) : u[r][j];
          } else {
            A[j] *= al[r][j];
            B[j] = kDown ? al[r][j] * (B[j] + v[j]) : fmaf(al[r][j], B[j], u[r][j]);
          }
        }
      }
    };
    if (edge)
      reduce(std::true_type{});
    else
      reduce(std::false_type{});
    *reinterpret_cast<float4*>(&sh.pair[warp][0][lane * 4]) = make_float4(A[0], A[1], A[2], A[3]);
    *reinterpret_cast<float4*>(&sh.pair[warp][1][lane * 4]) = make_float4(B[0], B[1], B[2], B[3]);
    __syncthreads();  // the pairs are there, and every warp is done with the tile before

    // ---- what enters each warp's rows: one thread per channel
    const int place = chunk % kGroup;
    if (warp < kBlock / 32) {
      const int ch = threadIdx.x;
      float* pairs = p.pairs + ((size_t)chain * p.chunks + chunk) * (2 * kBlock) + ch;
      if (!p.in_order && place != kGroup - 1 && chunk != p.chunks - 1) {
        float ta = sh.pair[0][0][ch], tb = sh.pair[0][1][ch];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const float wa = sh.pair[w][0][ch], wb = sh.pair[w][1][ch];
          tb = through(tb, wa, wb);
          ta = fresh(wa) ? wa : ta * wa;
        }
        publish(pairs, ta);
        publish(pairs + kBlock, tb);
      }
      float h = 0.f;
      if (p.in_order) {
        if (chunk > 0) h = sh.carry[ch];
      } else {
        auto arrived = [&](const float* q, uint32_t v) {
          for (uint32_t i = 0; v == kEmpty; ++i) {
            if (i >= (failed ? 1u : kPollLimit)) {
              failed = true;
              gave_up(203);
              break;
            }
            v = peek(q);
          }
          return __uint_as_float(v);
        };
        const float* head = p.states + ((size_t)chain * p.groups + chunk / kGroup - 1) * kBlock + ch;
        uint32_t hv = 0, va[kGroup - 1], vb[kGroup - 1];
        if (chunk >= kGroup) hv = peek(head);
        const float* q = pairs - (size_t)place * (2 * kBlock);
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k)
          if (k < place) va[k] = peek(q + k * 2 * kBlock), vb[k] = peek(q + (k * 2 + 1) * kBlock);
        if (chunk >= kGroup) h = arrived(head, hv);
#pragma unroll
        for (int k = 0; k < kGroup - 1; ++k)
          if (k < place) {
            const float ka = arrived(q + k * 2 * kBlock, va[k]), kb = arrived(q + (k * 2 + 1) * kBlock, vb[k]);
            h = through(h, ka, kb);
          }
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        sh.enter[w][ch] = h;
        h = through(h, sh.pair[w][0][ch], sh.pair[w][1][ch]);
      }
      if (p.in_order)
        sh.carry[ch] = h;
      else if (place == kGroup - 1)
        publish(p.states + ((size_t)chain * p.groups + chunk / kGroup) * kBlock + ch, h);
    } else if (warp == kFeeder) {
      feed(it + 2);  // into the stage of the tile before this one
    }
    __syncthreads();
    float h[4];  // the state that enters (forward), c_{t+1} (backward)
    {
      const float4 q = *reinterpret_cast<const float4*>(&sh.enter[warp][lane * 4]);
      h[0] = q.x, h[1] = q.y, h[2] = q.z, h[3] = q.w;
    }

    // ---- the rows themselves
    int lam_code = 0, z_code = 0;  // of row `lane` of the warp
    auto emit = [&](auto edges) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = row_at(r);
        const Row q = edges.value ? row_info(i) : Row{true, false, false, 0};
        if (edges.value && !q.valid) {
          if (packed && t0 + i < a.T) {  // a row that no sequence owns
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            stg4(static_cast<IO*>(a.out) + global_row(i) * a.D + c, zero, n, p.vec);
            if (kDown) stg4(static_cast<IO*>(a.dg) + global_row(i) * a.D + c, zero, n, p.vec);
            if (kSave) {
              const ScanCkptLayout l = scan_ckpt_layout(rows, a.D);
              if (n > 0) {
                *reinterpret_cast<uint32_t*>(a.ckpt + global_row(i) * l.pitch + c) = 0;
                *reinterpret_cast<uint32_t*>(a.ckpt + l.z + global_row(i) * l.pitch + c) = 0;
              }
              if (lane == r) lam_code = z_code = 1;
            }
          }
          continue;
        }
        const bool start = edges.value && (kDown ? q.last : q.first);
        if constexpr (!kDown) {
          float z[4], lam[4];
          if constexpr (kSave) {
            float g[4];
            load_gate(i, g);
            if (start)
              state_of(a.s0, q.seq, z);
            else
#pragma unroll
              for (int j = 0; j < 4; ++j) z[j] = h[j];
            if (COMPL) {
              float x[4];
              lds4<IO>(elem(0, i), x);
#pragma unroll
              for (int j = 0; j < 4; ++j) z[j] -= x[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) lam[j] = !RAW ? g[j] : j < n ? log_sigmoid(g[j]) : 0.f;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = start ? u[r][j] : fmaf(al[r][j], h[j], u[r][j]);
          stg4(static_cast<IO*>(a.out) + global_row(i) * a.D + c, h, n, p.vec);
          if constexpr (kSave) {
            const ScanCkptLayout l = scan_ckpt_layout(rows, a.D);
            uint32_t ml = 0, mz = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) ml = max(ml, magnitude(lam[j])), mz = max(mz, magnitude(z[j]));
            const int kl = scale_code(__uint_as_float(__reduce_max_sync(0xffffffffu, ml)));
            const int kz = scale_code(__uint_as_float(__reduce_max_sync(0xffffffffu, mz)));
            if (n > 0) {
              *reinterpret_cast<uint32_t*>(a.ckpt + global_row(i) * l.pitch + c) = encode4(lam, pow2(254 - kl));
              *reinterpret_cast<uint32_t*>(a.ckpt + l.z + global_row(i) * l.pitch + c) = encode4(z, pow2(254 - kz));
            }
            if (lane == r) lam_code = kl, z_code = kz;
          }
          if (edges.value && q.last && a.sT) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < n) a.sT[(size_t)q.seq * a.D + c + j] = h[j];
          }
        } else {
          float z[4], v[4], dx[4], dg[4], from[4];
          lds4<IO>(elem(0, i), v);
          if (start) state_of(a.s0, q.seq, from);
          if constexpr (kFrom) {
            decode4(*reinterpret_cast<const uint32_t*>(elem(2, i)), pow2(sh.scale[s][1][i]), z);
          } else {
            if (edges.value && q.first)
              state_of(a.h0, q.seq, z);
            else
              lds4<IO>(elem(2, i), z);
            if (COMPL) {
              float x[4];
              lds4<IO>(elem(3, i), x);
#pragma unroll
              for (int j = 0; j < 4; ++j) z[j] -= x[j];
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float d = v[j] + (start ? from[j] : h[j]);
            h[j] = al[r][j] * d;
            dx[j] = COMPL ? u[r][j] * d : d;
            dg[j] = RAW ? h[j] * z[j] * u[r][j] : h[j] * z[j];
          }
          stg4(static_cast<IO*>(a.out) + global_row(i) * a.D + c, dx, n, p.vec);
          stg4(static_cast<IO*>(a.dg) + global_row(i) * a.D + c, dg, n, p.vec);
          if (edges.value && q.first && a.sT) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < n) a.sT[(size_t)q.seq * a.D + c + j] = h[j];
          }
        }
      }
      if (kSave && lane < R && t0 + warp * R + lane < a.T) {
        const ScanCkptLayout l = scan_ckpt_layout(rows, a.D);
        const size_t at = cb * rows + global_row(warp * R + lane);
        a.ckpt[l.lam_scale + at] = (uint8_t)lam_code;
        a.ckpt[l.z_scale + at] = (uint8_t)z_code;
      }
    };
    if (edge)
      emit(std::true_type{});
    else
      emit(std::false_type{});
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
  for (size_t t = at; t < (size_t)a.T; t += step) {
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
    lds4<IO>(reinterpret_cast<const uint8_t*>(g + i), gv);
    lds4<IO>(reinterpret_cast<const uint8_t*>(x + i), xv);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) gv[j] = j < n ? to_f32(g[i + j]) : 0.f, xv[j] = j < n ? to_f32(x[i + j]) : 0.f;
  }
  ldg4(state + i, s, n, n == 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float alpha, beta;
    gate<RAW>(gv[j], alpha, beta);
    s[j] = fmaf(alpha, s[j], COMPL ? beta * xv[j] : xv[j]);
  }
  stg4(out_state + i, s, n, n == 4);
  stg4(h + i, s, n, n == 4);
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

// [B][T][row of `pitch` elements, `width` of them read]; box 128 channels x `box_rows` rows.
bool make_map(CUtensorMap* map, const void* base, int eb, int B, int T, size_t width, size_t pitch, int box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  const CUtensorMapDataType type = eb == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : eb == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  cuuint64_t dims[3] = {width, (cuuint64_t)T, (cuuint64_t)B};
  cuuint64_t strides[2] = {pitch * eb, pitch * eb * (cuuint64_t)T};
  cuuint32_t box[3] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
  return enc(map, type, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMinRows = kWarps * 4;  // of a tile, over all kinds

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, bool after,
                   const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr, cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <Kind K, typename IO, bool RAW, bool COMPL>
cudaError_t launch_tiles(const ScanArgs& a, void* ws, cudaStream_t stream) {
  using S = Shape<K, IO, COMPL>;
  TileArgs p;
  p.a = a;
  p.blocks = (int)div_up(a.D, kBlock);
  const int64_t chains = (int64_t)a.B * p.blocks, chunks = div_up(a.T, S::kL);
  p.chains = (int)chains, p.chunks = (int)chunks, p.groups = (int)div_up(chunks, kGroup);
  p.in_order = a.T <= kInOrderRows;
  p.vec = a.D % 4 == 0;
  p.tma = (size_t)a.D * sizeof(IO) % 16 == 0;
  // workspace: header, pairs, states, row information (the last two kinds of words only where needed)
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.hdr = reinterpret_cast<WorkspaceHeader*>(w);
  w += sizeof(WorkspaceHeader);
  p.pairs = reinterpret_cast<float*>(w);
  const size_t pair_words = p.in_order ? 0 : (size_t)(chains * chunks) * (2 * kBlock);
  const size_t state_words = p.in_order ? 0 : (size_t)chains * p.groups * kBlock;
  p.states = p.pairs + pair_words;
  int32_t* info = reinterpret_cast<int32_t*>(p.states + state_words);
  p.info = info;
  if (!ws || (p.in_order && !a.cu)) p.hdr = nullptr;  // no workspace
  if (p.tma) {
    const int eb = sizeof(IO);
    const size_t d = (size_t)a.D;
    bool ok;
    if (K == kFwd || K == kFwdCkpt) {
      ok = make_map(&p.map[0], a.x, eb, a.B, a.T, d, d, S::kL) && make_map(&p.map[1], a.g, eb, a.B, a.T, d, d, S::kL);
    } else if (K == kBwd) {
      ok = make_map(&p.map[0], a.dy, eb, a.B, a.T, d, d, S::kL) && make_map(&p.map[1], a.g, eb, a.B, a.T, d, d, S::kL) &&
           make_map(&p.map[2], a.h, eb, a.B, a.T, d, d, S::kL) &&
           (!COMPL || make_map(&p.map[3], a.x, eb, a.B, a.T, d, d, S::kL));
    } else {
      const ScanCkptLayout l = scan_ckpt_layout((size_t)a.B * a.T, a.D);
      ok = make_map(&p.map[0], a.dy, eb, a.B, a.T, d, d, S::kL) &&
           make_map(&p.map[1], a.ckpt, 1, a.B, a.T, d, l.pitch, S::kL) &&
           make_map(&p.map[2], a.ckpt + l.z, 1, a.B, a.T, d, l.pitch, S::kL);
    }
    if (!ok) return cudaErrorInvalidValue;
  }
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
  const int sms = sm_count();
  const bool init = !p.in_order || a.cu;
  if (init) {
    const size_t count = (pair_words + state_words) / 4;
    const int64_t blocks = std::min<int64_t>(std::max<int64_t>(div_up((int64_t)count, 256 * 4), div_up(a.cu ? a.T : 1, 256)), sms * 8);
    e = launch(scan_init_kernel, (unsigned)std::max<int64_t>(blocks, 1), 256, 0, stream, false, p,
               reinterpret_cast<uint4*>(p.pairs), count, info);
    if (e != cudaSuccess) return e;
  }
  const int64_t grid = p.in_order ? chains : std::min<int64_t>(chains * chunks, (int64_t)sms * S::kPerSm);
  return launch(kernel, (unsigned)grid, 32 * kWarps, S::kSmem, stream, init, p);
}

}  // namespace

// Enough for every kind of call: the forward and the backward of a type share one size.
size_t scan_workspace_bytes(int B, int T, int D, int N, int dtype) {
  (void)dtype;
  if (B == 0 || T == 0) return 0;
  const int64_t chains = (int64_t)B * div_up(D, kBlock), chunks = div_up(T, kMinRows);
  size_t bytes = 0;
  if (T > kInOrderRows)
    bytes = (size_t)(chains * (2 * chunks + div_up(chunks, kGroup))) * kBlock * sizeof(float);
  if (N > 0) bytes += align256((size_t)T * 4);
  return bytes ? sizeof(WorkspaceHeader) + bytes : 0;
}

cudaError_t launch_scan_fwd(const ScanArgs& a, void* ws, cudaStream_t stream) {
  return with_flags(a.dtype, a.prep, a.complement, [&](auto io, auto raw, auto compl_) {
    return a.ckpt ? launch_tiles<kFwdCkpt, decltype(io), raw.value, compl_.value>(a, ws, stream)
                  : launch_tiles<kFwd, decltype(io), raw.value, compl_.value>(a, ws, stream);
  });
}

cudaError_t launch_scan_bwd(const ScanArgs& a, void* ws, cudaStream_t stream) {
  return with_flags(a.dtype, a.prep, a.complement, [&](auto io, auto raw, auto compl_) {
    return a.ckpt ? launch_tiles<kBwdCkpt, decltype(io), raw.value, compl_.value>(a, ws, stream)
                  : launch_tiles<kBwd, decltype(io), raw.value, compl_.value>(a, ws, stream);
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
