// kda_scan.cu -- elementwise gated linear recurrence: sequences, backward, step.
//
//     h_t = alpha_t h_{t-1} + w_t x_t,   alpha_t = exp(lambda_t),   w_t = 1 or 1 - alpha_t
//
// lambda_t is the given log-gate or log sigmoid of a raw projection.  One
// thread per channel walks its sequence; a block holds 128 channels, which
// are one scale block of the 8-bit checkpoint.
#include <cuda_fp8.h>

#include <type_traits>

#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int kBlock = 128;  // channels per scale of the checkpoint, and threads per block

// alpha and 1 - alpha, each to a few ulp on its own (1 - alpha by subtraction
// would lose the small rates that make the long memories), and, where asked
// for, lambda.
template <bool RAW>
__device__ __forceinline__ void gate(float g, float& alpha, float& beta) {
  if (RAW) {
    const float e = expf(-fabsf(g)), inv = __frcp_rn(1.f + e), lo = e * inv;
    alpha = g >= 0.f ? inv : lo;
    beta = g >= 0.f ? lo : inv;
  } else {
    alpha = expf(g);
    beta = -expm1f(g);
  }
}

template <typename T>
__device__ __forceinline__ float load(const T* p, size_t i) { return to_f32(__ldg(p + i)); }

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
__device__ __forceinline__ uint8_t encode(float v, float inv) {
  v = fabsf(v) <= 3.402823466e38f ? v * inv : __int_as_float(0x7fffffff);
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float decode(uint8_t c, float scale) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3))) * scale;
}

// The block's maximum magnitude (bits), over its 128 threads.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* buf) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return max(max(buf[0], buf[1]), max(buf[2], buf[3]));
}

// The rows [lo, hi) of sequence s, clamped to the buffer.
__device__ __forceinline__ void rows_of(const ScanArgs& a, int s, int64_t& lo, int64_t& hi) {
  if (a.cu) {
    lo = min(max(__ldg(a.cu + s), 0), a.T);
    hi = min(max(__ldg(a.cu + s + 1), 0), a.T);
  } else {
    lo = (int64_t)s * a.T;
    hi = lo + a.T;
  }
}

// Zeros in the rows that no sequence owns (packed only).
template <typename IO>
__device__ void zero_rows(const ScanArgs& a, int c, int64_t lo, int64_t hi) {
  const ScanCkptLayout l = scan_ckpt_layout((size_t)a.B * a.T, a.D);
  for (int64_t t = lo; t < hi; ++t) {
    if (c < a.D) {
      static_cast<IO*>(a.out)[(size_t)t * a.D + c] = from_f32<IO>(0.f);
      if (a.dg) static_cast<IO*>(a.dg)[(size_t)t * a.D + c] = from_f32<IO>(0.f);
      if (a.ckpt && !a.dy) a.ckpt[t * l.pitch + c] = a.ckpt[l.z + t * l.pitch + c] = 0;
    }
    if (a.ckpt && !a.dy && threadIdx.x == 0) {
      const size_t at = (size_t)blockIdx.x * a.B * a.T + t;
      a.ckpt[l.lam_scale + at] = a.ckpt[l.z_scale + at] = 1;
    }
  }
}

template <typename IO, bool RAW, bool COMPL>
__global__ void __launch_bounds__(kBlock) scan_fwd_kernel(const ScanArgs a) {
  __shared__ uint32_t red[2][4];
  const int c = blockIdx.x * kBlock + threadIdx.x, nseq = a.cu ? a.N : a.B;
  const bool live = c < a.D;
  const size_t rows = (size_t)a.B * a.T;
  const ScanCkptLayout l = scan_ckpt_layout(rows, a.D);
  for (int s = blockIdx.y; s < nseq; s += gridDim.y) {
    int64_t lo, hi;
    rows_of(a, s, lo, hi);
    const size_t st = (size_t)s * a.D + c;
    float h = live && a.s0 ? a.s0[st] : 0.f;
    for (int64_t t = lo; t < hi; ++t) {
      const size_t at = (size_t)t * a.D + c;
      const float g = live ? load(static_cast<const IO*>(a.g), at) : 0.f;
      const float x = live ? load(static_cast<const IO*>(a.x), at) : 0.f;
      float alpha, beta;
      gate<RAW>(g, alpha, beta);
      if (a.ckpt) {
        const float lam = RAW ? log_sigmoid(g) : g, z = COMPL ? h - x : h;
        const int kl = scale_code(__uint_as_float(block_max(live ? magnitude(lam) : 0u, red[0])));
        const int kz = scale_code(__uint_as_float(block_max(live ? magnitude(z) : 0u, red[1])));
        if (live) {
          a.ckpt[t * l.pitch + c] = encode(lam, pow2(254 - kl));
          a.ckpt[l.z + t * l.pitch + c] = encode(z, pow2(254 - kz));
        }
        if (threadIdx.x == 0) {
          a.ckpt[l.lam_scale + blockIdx.x * rows + t] = (uint8_t)kl;
          a.ckpt[l.z_scale + blockIdx.x * rows + t] = (uint8_t)kz;
        }
      }
      h = fmaf(alpha, h, COMPL ? beta * x : x);
      if (live) static_cast<IO*>(a.out)[at] = from_f32<IO>(h);
    }
    if (live && a.sT) a.sT[st] = h;
    if (a.cu) {
      if (s == 0) zero_rows<IO>(a, c, 0, lo);
      if (s == nseq - 1) zero_rows<IO>(a, c, hi, a.T);
    }
  }
}

template <typename IO, bool RAW, bool COMPL>
__global__ void __launch_bounds__(kBlock) scan_bwd_kernel(const ScanArgs a) {
  const int c = blockIdx.x * kBlock + threadIdx.x, nseq = a.cu ? a.N : a.B;
  if (c >= a.D) return;
  const size_t rows = (size_t)a.B * a.T;
  const ScanCkptLayout l = scan_ckpt_layout(rows, a.D);
  for (int s = blockIdx.y; s < nseq; s += gridDim.y) {
    int64_t lo, hi;
    rows_of(a, s, lo, hi);
    const size_t st = (size_t)s * a.D + c;
    float carry = a.s0 ? a.s0[st] : 0.f;
    for (int64_t t = hi - 1; t >= lo; --t) {
      const size_t at = (size_t)t * a.D + c;
      float alpha, beta, z;
      if (a.ckpt) {
        gate<false>(decode(a.ckpt[t * l.pitch + c], pow2(a.ckpt[l.lam_scale + blockIdx.x * rows + t])), alpha, beta);
        z = decode(a.ckpt[l.z + t * l.pitch + c], pow2(a.ckpt[l.z_scale + blockIdx.x * rows + t]));
      } else {
        gate<RAW>(load(static_cast<const IO*>(a.g), at), alpha, beta);
        z = t > lo ? load(static_cast<const IO*>(a.h), at - a.D) : a.h0 ? a.h0[st] : 0.f;
        if (COMPL) z -= load(static_cast<const IO*>(a.x), at);
      }
      const float d = load(static_cast<const IO*>(a.dy), at) + carry;
      carry = alpha * d;
      static_cast<IO*>(a.out)[at] = from_f32<IO>(COMPL ? beta * d : d);
      static_cast<IO*>(a.dg)[at] = from_f32<IO>(RAW ? carry * z * beta : carry * z);
    }
    if (a.sT) a.sT[st] = carry;
    if (a.cu) {
      if (s == 0) zero_rows<IO>(a, c, 0, lo);
      if (s == nseq - 1) zero_rows<IO>(a, c, hi, a.T);
    }
  }
}

template <typename IO, bool RAW, bool COMPL>
__global__ void __launch_bounds__(256) scan_step_kernel(const IO* __restrict__ x, const IO* __restrict__ g,
                                                        const float* state, float* out_state, IO* __restrict__ h,
                                                        size_t n) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float alpha, beta;
  gate<RAW>(to_f32(g[i]), alpha, beta);
  const float v = to_f32(x[i]), r = fmaf(alpha, state[i], COMPL ? beta * v : v);
  out_state[i] = r;
  h[i] = from_f32<IO>(r);
}

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

dim3 scan_grid(const ScanArgs& a) {
  const int nseq = a.cu ? a.N : a.B;
  return dim3((unsigned)((a.D + kBlock - 1) / kBlock), (unsigned)(nseq < 65535 ? nseq : 65535));
}

}  // namespace

size_t scan_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_scan_fwd(const ScanArgs& a, void*, cudaStream_t stream) {
  return with_flags(a.dtype, a.prep, a.complement, [&](auto io, auto raw, auto compl_) {
    scan_fwd_kernel<decltype(io), raw.value, compl_.value><<<scan_grid(a), kBlock, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

cudaError_t launch_scan_bwd(const ScanArgs& a, void*, cudaStream_t stream) {
  return with_flags(a.dtype, a.prep, a.complement, [&](auto io, auto raw, auto compl_) {
    scan_bwd_kernel<decltype(io), raw.value, compl_.value><<<scan_grid(a), kBlock, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

cudaError_t launch_scan_step(const void* x, const void* g, const float* state, float* out_state, void* h, size_t n,
                             int dtype, int prep, int complement, cudaStream_t stream) {
  return with_flags(dtype, prep, complement, [&](auto io, auto raw, auto compl_) {
    using IO = decltype(io);
    scan_step_kernel<IO, raw.value, compl_.value><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(
        static_cast<const IO*>(x), static_cast<const IO*>(g), state, out_state, static_cast<IO*>(h), n);
    return cudaGetLastError();
  });
}

}  // namespace kda
