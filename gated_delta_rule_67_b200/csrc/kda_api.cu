// kda_api.cu -- the C ABI of libkda.so: host-side validation and dispatch.
//
// Every argument is checked here, before anything is enqueued; the kernels
// themselves assume valid, aligned, non-overlapping buffers.
#include <string.h>

#include "kda_common.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
  const char* lo;
  size_t bytes;
};

bool overlaps(Range a, Range b) {
  if (!a.lo || !b.lo || a.bytes == 0 || b.bytes == 0) return false;
  return a.lo < b.lo + b.bytes && b.lo < a.lo + a.bytes;
}

size_t elem_bytes(int dtype) { return dtype == KDA_F32 ? 4 : 2; }

kda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

bool prefill_supported(int dk, int dv, int chunk, int dtype) {
  if (dtype == KDA_F32)
    return (dk == 64 || dk == 128) && (dv == 64 || dv == 128) &&
           (chunk == 16 || chunk == 32 || chunk == 64);
  return (dk == 64 || dk == 128) && (dv == 64 || dv == 128) && chunk == 64;
}

}  // namespace

extern "C" {

const char* kda_status_string(int status) {
  switch (status) {
    case KDA_OK: return "KDA_OK";
    case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG: null, misaligned, overlapping or out-of-range argument";
    case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED: valid arguments outside the implemented shapes/dtypes";
    case KDA_ERR_CUDA: return "KDA_ERR_CUDA: a CUDA runtime call or kernel launch failed";
    case KDA_ERR_TIMEOUT: return "KDA_ERR_TIMEOUT: a bounded on-device wait gave up";
    default: return "KDA_ERR_UNKNOWN: not a kda_status value";
  }
}

int kda_version(void) { return 100; }

size_t kda_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int chunk, int dtype) {
  if (B < 0 || T < 0 || H < 1 || dk < 1 || dv < 1 || chunk < 1) return 0;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
  if (!prefill_supported(dk, dv, chunk, dtype)) return 0;
  if (dtype == KDA_BF16) return kda::prefill_bf16_workspace_bytes(B, T, H, dk, dv, chunk);
  return 0;
}

int kda_chunk_fwd_launch_count(int B, int T, int H, int dk, int dv, int chunk, int dtype) {
  if (B < 0 || T < 0 || H < 1 || dk < 1 || dv < 1 || chunk < 1) return -1;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return -1;
  if (!prefill_supported(dk, dv, chunk, dtype)) return -1;
  if (B == 0 || T == 0) return 0;
  return dtype == KDA_BF16 ? kda::prefill_bf16_launches(B, T, H) : 1;
}

static kda_status chunk_fwd_impl(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                 float scale, const float* initial_state, void* o, float* final_state, int B,
                                 int T, int H, int dk, int dv, int chunk, int dtype, int gate, int prep,
                                 void* workspace, size_t workspace_bytes, void* stream_, void* const* events) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (B < 0 || T < 0 || H < 1 || dk < 1 || dv < 1 || chunk < 1) return KDA_ERR_INVALID_ARG;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (gate != KDA_GATE_CHANNEL && gate != KDA_GATE_HEAD && gate != KDA_GATE_NONE) return KDA_ERR_INVALID_ARG;
  if (prep & ~kda::kPrepMask) return KDA_ERR_INVALID_ARG;
  if (gate == KDA_GATE_NONE) g = nullptr;
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return KDA_ERR_INVALID_ARG;
  const bool empty = (B == 0 || T == 0);
  const size_t eb = elem_bytes(dtype);
  const size_t ntok = (size_t)B * T * H;
  const Range rq{(const char*)q, ntok * dk * eb}, rk{(const char*)k, ntok * dk * eb},
      rg{(const char*)g, gate == KDA_GATE_CHANNEL ? ntok * dk * eb : ntok * eb}, rv{(const char*)v, ntok * dv * eb},
      rb{(const char*)beta, ntok * eb}, ro{(const char*)o, ntok * dv * eb};
  const size_t state_bytes = (size_t)B * H * dk * dv * sizeof(float);
  const Range rs0{(const char*)initial_state, state_bytes}, rsT{(const char*)final_state, state_bytes};
  if (!empty) {
    const void* need[] = {q, k, v, o};
    for (const void* p : need)
      if (!p || !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (!beta || !aligned_to(beta, eb)) return KDA_ERR_INVALID_ARG;
    if (gate == KDA_GATE_CHANNEL && (!g || !aligned16(g))) return KDA_ERR_INVALID_ARG;
    if (gate == KDA_GATE_HEAD && (!g || !aligned_to(g, eb))) return KDA_ERR_INVALID_ARG;
    // o is written: it must not overlap any input.
    for (Range r : {rq, rk, rg, rv, rb, rs0})
      if (overlaps(ro, r)) return KDA_ERR_INVALID_ARG;
  }
  if (initial_state && !aligned16(initial_state)) return KDA_ERR_INVALID_ARG;
  if (final_state && !aligned16(final_state)) return KDA_ERR_INVALID_ARG;
  if (final_state && !empty) {
    for (Range r : {rq, rk, rg, rv, rb, ro})
      if (overlaps(rsT, r)) return KDA_ERR_INVALID_ARG;
    if (initial_state && (const void*)initial_state != (const void*)final_state && overlaps(rsT, rs0))
      return KDA_ERR_INVALID_ARG;
  }
  if (!prefill_supported(dk, dv, chunk, dtype)) return KDA_ERR_UNSUPPORTED;
  const size_t need_ws = kda_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, dtype);
  if (need_ws > 0 && !empty) {
    if (!workspace || workspace_bytes < need_ws || (reinterpret_cast<uintptr_t>(workspace) & 255u))
      return KDA_ERR_INVALID_ARG;
    const Range rw{(const char*)workspace, workspace_bytes};
    for (Range r : {rq, rk, rg, rv, rb, ro, rs0, rsT})
      if (overlaps(rw, r)) return KDA_ERR_INVALID_ARG;
  }

  if (events)
    for (int i = 0; i < 3; ++i)
      if (!events[i]) return KDA_ERR_INVALID_ARG;
  if (empty) {
    // Nothing to run: the final state is the initial state (or zeros).
    cudaError_t e = cudaSuccess;
    if (final_state && state_bytes && initial_state != final_state)
      e = initial_state ? cudaMemcpyAsync(final_state, initial_state, state_bytes, cudaMemcpyDeviceToDevice, stream)
                        : cudaMemsetAsync(final_state, 0, state_bytes, stream);
    for (int i = 0; i < 3 && e == cudaSuccess; ++i) e = kda::mark(events, i, stream);
    return from_cuda(e);
  }

  cudaError_t e;
  if (dtype == KDA_F32) {
    e = kda::launch_prefill_f32((const float*)q, (const float*)k, (const float*)v, (const float*)g,
                                (const float*)beta, scale, initial_state, (float*)o, final_state, B, T,
                                H, dk, dv, chunk, gate, prep, stream, events);
  } else {
    e = kda::launch_prefill_bf16((const __nv_bfloat16*)q, (const __nv_bfloat16*)k,
                                 (const __nv_bfloat16*)v, (const __nv_bfloat16*)g,
                                 (const __nv_bfloat16*)beta, scale, initial_state, (__nv_bfloat16*)o,
                                 final_state, B, T, H, dk, dv, chunk, gate, prep, workspace, workspace_bytes,
                                 stream, events);
  }
  return from_cuda(e);
}

kda_status kda_chunk_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                         float scale, const float* initial_state, void* o, float* final_state, int B,
                         int T, int H, int dk, int dv, int chunk, int dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return chunk_fwd_impl(q, k, v, g, beta, scale, initial_state, o, final_state, B, T, H, dk, dv, chunk, dtype,
                        KDA_GATE_CHANNEL, KDA_PREP_NONE, workspace, workspace_bytes, stream, nullptr);
}

kda_status kda_chunk_fwd_ex(const void* q, const void* k, const void* v, const void* g, const void* beta,
                            float scale, const float* initial_state, void* o, float* final_state, int B, int T,
                            int H, int dk, int dv, int chunk, int dtype, int gate, int prep, void* workspace,
                            size_t workspace_bytes, void* stream) {
  return chunk_fwd_impl(q, k, v, g, beta, scale, initial_state, o, final_state, B, T, H, dk, dv, chunk, dtype,
                        gate, prep, workspace, workspace_bytes, stream, nullptr);
}

kda_status kda_chunk_fwd_profiled(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                  float scale, const float* initial_state, void* o, float* final_state, int B,
                                  int T, int H, int dk, int dv, int chunk, int dtype, void* workspace,
                                  size_t workspace_bytes, void* stream, void* const* events) {
  if (!events) return KDA_ERR_INVALID_ARG;
  return chunk_fwd_impl(q, k, v, g, beta, scale, initial_state, o, final_state, B, T, H, dk, dv, chunk, dtype,
                        KDA_GATE_CHANNEL, KDA_PREP_NONE, workspace, workspace_bytes, stream, events);
}

kda_status kda_chunk_fwd_check(const void* workspace, size_t workspace_bytes, void* stream_) {
  if (!workspace || workspace_bytes < sizeof(kda::WorkspaceHeader)) return KDA_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  kda::WorkspaceHeader h;
  cudaError_t e = cudaMemcpyAsync(&h, workspace, sizeof(h), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  return h.error ? KDA_ERR_TIMEOUT : KDA_OK;
}

kda_status kda_wait_selftest(void* workspace, size_t workspace_bytes, void* stream_) {
  if (!workspace || workspace_bytes < sizeof(kda::WorkspaceHeader) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return KDA_ERR_INVALID_ARG;
  return from_cuda(kda::launch_wait_selftest(workspace, static_cast<cudaStream_t>(stream_)));
}

size_t kda_backward_workspace_size(int B, int T, int H, int dk, int dv, int dtype) {
  if (B < 0 || T < 0 || H < 1) return 0;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return 0;
  if (!((dk == 64 || dk == 128) && (dv == 64 || dv == 128))) return 0;
  return kda::backward_workspace_bytes(B, T, H, dk, dv, dtype);
}

size_t kda_backward_ex_workspace_size(int B, int T, int H, int dk, int dv, int dtype, int prep) {
  const size_t base = kda_backward_workspace_size(B, T, H, dk, dv, dtype);
  if (base == 0 || (prep & ~kda::kPrepMask)) return 0;
  return prep ? base + kda::backward_prep_bytes(B, T, H, dk, dtype) : base;
}

kda_status kda_backward(const void* q, const void* k, const void* v, const void* g, const void* beta, float scale,
                        const float* initial_state, const void* grad_o, const float* grad_final_state, void* grad_q,
                        void* grad_k, void* grad_v, void* grad_g, void* grad_beta, float* grad_initial_state, int B,
                        int T, int H, int dk, int dv, int dtype, int gate, void* workspace, size_t workspace_bytes,
                        void* stream_) {
  return kda_backward_ex(q, k, v, g, beta, scale, initial_state, grad_o, grad_final_state, grad_q, grad_k, grad_v,
                         grad_g, grad_beta, grad_initial_state, B, T, H, dk, dv, dtype, gate, KDA_PREP_NONE, workspace,
                         workspace_bytes, stream_);
}

kda_status kda_backward_ex(const void* q, const void* k, const void* v, const void* g, const void* beta, float scale,
                           const float* initial_state, const void* grad_o, const float* grad_final_state, void* grad_q,
                           void* grad_k, void* grad_v, void* grad_g, void* grad_beta, float* grad_initial_state, int B,
                           int T, int H, int dk, int dv, int dtype, int gate, int prep, void* workspace,
                           size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (B < 0 || T < 0 || H < 1 || dk < 1 || dv < 1) return KDA_ERR_INVALID_ARG;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (gate != KDA_GATE_CHANNEL && gate != KDA_GATE_HEAD && gate != KDA_GATE_NONE) return KDA_ERR_INVALID_ARG;
  if (prep & ~kda::kPrepMask) return KDA_ERR_INVALID_ARG;
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return KDA_ERR_INVALID_ARG;
  if (gate == KDA_GATE_NONE) g = nullptr, grad_g = nullptr;
  const bool empty = (B == 0 || T == 0);
  const size_t eb = elem_bytes(dtype), ntok = (size_t)B * T * H, state_bytes = (size_t)B * H * dk * dv * 4;
  const size_t gbytes = gate == KDA_GATE_CHANNEL ? ntok * dk * eb : ntok * eb;
  const Range rq{(const char*)q, ntok * dk * eb}, rk{(const char*)k, ntok * dk * eb},
      rv{(const char*)v, ntok * dv * eb}, rg{(const char*)g, gbytes}, rb{(const char*)beta, ntok * eb},
      rs0{(const char*)initial_state, state_bytes}, rdo{(const char*)grad_o, ntok * dv * eb},
      rdsT{(const char*)grad_final_state, state_bytes};
  const Range wq{(const char*)grad_q, ntok * dk * eb}, wk{(const char*)grad_k, ntok * dk * eb},
      wv{(const char*)grad_v, ntok * dv * eb}, wg{(const char*)grad_g, gbytes}, wb{(const char*)grad_beta, ntok * eb},
      ws0{(const char*)grad_initial_state, state_bytes};
  if (!empty) {
    const void* need[] = {q, k, v, grad_o, grad_q, grad_k, grad_v};
    for (const void* p : need)
      if (!p || !aligned16(p)) return KDA_ERR_INVALID_ARG;
    for (const void* p : {beta, (const void*)grad_beta})
      if (!p || !aligned_to(p, eb)) return KDA_ERR_INVALID_ARG;
    if (gate == KDA_GATE_CHANNEL && (!g || !grad_g || !aligned16(g) || !aligned16(grad_g))) return KDA_ERR_INVALID_ARG;
    if (gate == KDA_GATE_HEAD && (!g || !grad_g || !aligned_to(g, eb) || !aligned_to(grad_g, eb)))
      return KDA_ERR_INVALID_ARG;
  }
  for (const void* p : {(const void*)initial_state, (const void*)grad_final_state, (const void*)grad_initial_state})
    if (p && !aligned16(p)) return KDA_ERR_INVALID_ARG;
  const Range outs[] = {wq, wk, wv, wg, wb, ws0};
  for (int i = 0; i < 6; ++i) {
    for (Range r : {rq, rk, rv, rg, rb, rs0, rdo, rdsT})
      if (overlaps(outs[i], r)) return KDA_ERR_INVALID_ARG;
    for (int j = i + 1; j < 6; ++j)
      if (overlaps(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
  }
  if (!((dk == 64 || dk == 128) && (dv == 64 || dv == 128))) return KDA_ERR_UNSUPPORTED;
  if (empty) {  // dL/dS_0 = dL/dS_T
    cudaError_t e = cudaSuccess;
    if (grad_initial_state && state_bytes)
      e = grad_final_state ? cudaMemcpyAsync(grad_initial_state, grad_final_state, state_bytes,
                                             cudaMemcpyDeviceToDevice, stream)
                           : cudaMemsetAsync(grad_initial_state, 0, state_bytes, stream);
    return from_cuda(e);
  }
  // at least one (sequence, head)'s records, after the prepared inputs when `prep` is set
  const size_t prep_ws = prep ? kda::backward_prep_bytes(B, T, H, dk, dtype) : 0;
  const size_t need_ws = prep_ws + kda::backward_workspace_bytes(1, T, 1, dk, dv, dtype);
  if (!workspace || workspace_bytes < need_ws || !aligned16(workspace)) return KDA_ERR_INVALID_ARG;
  const Range rw{(const char*)workspace, workspace_bytes};
  for (Range r : {rq, rk, rv, rg, rb, rs0, rdo, rdsT, wq, wk, wv, wg, wb, ws0})
    if (overlaps(rw, r)) return KDA_ERR_INVALID_ARG;
  if (prep)
    return from_cuda(kda::launch_backward_prepared(q, k, v, g, beta, scale, initial_state, grad_o, grad_final_state,
                                                   grad_q, grad_k, grad_v, grad_g, grad_beta, grad_initial_state, B,
                                                   T, H, dk, dv, dtype, gate, prep, workspace, workspace_bytes,
                                                   stream));
  return from_cuda(kda::launch_backward(q, k, v, g, beta, scale, initial_state, grad_o, grad_final_state, grad_q,
                                        grad_k, grad_v, grad_g, grad_beta, grad_initial_state, B, T, H, dk, dv, dtype,
                                        gate, workspace, workspace_bytes, stream));
}

static kda_status recurrent_step_impl(const void* q, const void* k, const void* v, const void* g,
                                      const void* beta, float scale, float* state, void* o, int N, int H, int dk,
                                      int dv, int dtype, int gate, int prep, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (N < 0 || H < 1 || dk < 1 || dv < 1) return KDA_ERR_INVALID_ARG;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (gate != KDA_GATE_CHANNEL && gate != KDA_GATE_HEAD && gate != KDA_GATE_NONE) return KDA_ERR_INVALID_ARG;
  if (prep & ~kda::kPrepMask) return KDA_ERR_INVALID_ARG;
  if (gate == KDA_GATE_NONE) g = nullptr;
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return KDA_ERR_INVALID_ARG;
  if (N == 0) return KDA_OK;
  const size_t eb = elem_bytes(dtype);
  const void* need[] = {q, k, v, state, o};
  for (const void* p : need)
    if (!p || !aligned16(p)) return KDA_ERR_INVALID_ARG;
  if (!beta || !aligned_to(beta, eb)) return KDA_ERR_INVALID_ARG;
  if (gate == KDA_GATE_CHANNEL && (!g || !aligned16(g))) return KDA_ERR_INVALID_ARG;
  if (gate == KDA_GATE_HEAD && (!g || !aligned_to(g, eb))) return KDA_ERR_INVALID_ARG;
  const size_t nh = (size_t)N * H;
  const Range rq{(const char*)q, nh * dk * eb}, rk{(const char*)k, nh * dk * eb},
      rg{(const char*)g, gate == KDA_GATE_CHANNEL ? nh * dk * eb : nh * eb}, rv{(const char*)v, nh * dv * eb},
      rb{(const char*)beta, nh * eb}, ro{(const char*)o, nh * dv * eb},
      rs{(const char*)state, nh * dk * dv * sizeof(float)};
  for (Range r : {rq, rk, rg, rv, rb, rs})
    if (overlaps(ro, r)) return KDA_ERR_INVALID_ARG;
  for (Range r : {rq, rk, rg, rv, rb})
    if (overlaps(rs, r)) return KDA_ERR_INVALID_ARG;
  if (!((dk == 64 || dk == 128) && (dv == 64 || dv == 128))) return KDA_ERR_UNSUPPORTED;
  return from_cuda(kda::launch_decode(q, k, v, g, beta, scale, state, o, N, H, dk, dv, dtype, gate, prep, stream));
}

kda_status kda_recurrent_step(const void* q, const void* k, const void* v, const void* g,
                              const void* beta, float scale, float* state, void* o, int N, int H,
                              int dk, int dv, int dtype, void* stream) {
  return recurrent_step_impl(q, k, v, g, beta, scale, state, o, N, H, dk, dv, dtype, KDA_GATE_CHANNEL,
                             KDA_PREP_NONE, stream);
}

kda_status kda_recurrent_step_ex(const void* q, const void* k, const void* v, const void* g,
                                 const void* beta, float scale, float* state, void* o, int N, int H,
                                 int dk, int dv, int dtype, int gate, int prep, void* stream) {
  return recurrent_step_impl(q, k, v, g, beta, scale, state, o, N, H, dk, dv, dtype, gate, prep, stream);
}

// ------------------------------------------------ elementwise gated linear recurrence

// Sizes the scan entry points take: B, T, N >= 0, D >= 1, at most 2^40
// elements (so that byte counts cannot wrap), 2^31 - 1 tiles of 64 rows x 16
// channels and 2^28 packed sequences.  Returns the status they give.
static kda_status scan_sizes(int64_t B, int64_t T, int64_t D, int64_t N, int dtype) {
  if (B < 0 || T < 0 || D < 1 || N < 0) return KDA_ERR_INVALID_ARG;
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (T > INT32_MAX - 4096) return KDA_ERR_UNSUPPORTED;  // row numbers of a last tile stay within 32 bits
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (B * D > kMost || N * D > kMost || (T > 0 && B * D > kMost / T)) return KDA_ERR_UNSUPPORTED;
  if (B * ((D + 15) / 16) * ((T + 63) / 64) > INT32_MAX || N > (1 << 28)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

size_t kda_scan_workspace_size_ex(int B, int T, int D, int num_seqs, int dtype, int checkpoint) {
  if (scan_sizes(B, T, D, num_seqs, dtype) != KDA_OK || (num_seqs > 0 && B != 1)) return 0;
  return kda::scan_workspace_bytes(B, T, D, num_seqs, dtype, checkpoint != 0);
}

size_t kda_scan_workspace_size(int B, int T, int D, int num_seqs, int dtype) {
  return kda_scan_workspace_size_ex(B, T, D, num_seqs, dtype, 0);
}

size_t kda_scan_checkpoint_size(int B, int T, int D) {
  if (scan_sizes(B, T, D, 0, KDA_BF16) != KDA_OK) return 0;
  return kda::scan_ckpt_layout((size_t)B * T, D).total;
}

// What the three sequence calls share: sizes, flags, the buffers (each with
// whether it must be given), overlaps, workspace.
static kda_status scan_checks(const kda::ScanArgs& a, const Range* in, int n_in, const Range* out,
                              int n_out, const Range* need, int n_need, void* workspace, size_t workspace_bytes) {
  for (int i = 0; i < n_need; ++i)
    if (need[i].bytes && !need[i].lo) return KDA_ERR_INVALID_ARG;
  for (int i = 0; i < n_in; ++i)
    if (in[i].lo && !aligned16(in[i].lo) && (const void*)in[i].lo != (const void*)a.cu) return KDA_ERR_INVALID_ARG;
  for (int i = 0; i < n_out; ++i) {
    if (out[i].lo && !aligned16(out[i].lo)) return KDA_ERR_INVALID_ARG;
    for (int j = 0; j < n_in; ++j) {
      // the forward's final state may take the initial state's place (the checkpoint's z
      // reads the initial state when other blocks may already write the final one)
      if (out[i].lo == (const char*)a.sT && in[j].lo == (const char*)a.s0 && a.sT == a.s0 && !a.dy && !a.ckpt) continue;
      if (overlaps(out[i], in[j])) return KDA_ERR_INVALID_ARG;
    }
    for (int j = i + 1; j < n_out; ++j)
      if (overlaps(out[i], out[j])) return KDA_ERR_INVALID_ARG;
  }
  // the checkpoint is written (by the forward: it has no dy) from states kept in the workspace
  const size_t need_ws = kda::scan_workspace_bytes(a.B, a.T, a.D, a.N, a.dtype, a.ckpt && !a.dy);
  if (need_ws) {
    if (!workspace || workspace_bytes < need_ws || (reinterpret_cast<uintptr_t>(workspace) & 255u))
      return KDA_ERR_INVALID_ARG;
    const Range rw{(const char*)workspace, workspace_bytes};
    for (int i = 0; i < n_in; ++i)
      if (overlaps(rw, in[i])) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < n_out; ++i)
      if (overlaps(rw, out[i])) return KDA_ERR_INVALID_ARG;
  }
  return KDA_OK;
}

static kda_status scan_flags(int64_t B, int64_t T, int64_t D, const int32_t* cu, int64_t num_seqs, int dtype, int prep,
                             int input_gate) {
  const kda_status st = scan_sizes(B, T, D, cu ? num_seqs : 0, dtype);
  if (st != KDA_OK) return st;
  if (prep & ~KDA_PREP_GATE_LOGSIGMOID) return KDA_ERR_INVALID_ARG;
  if (input_gate != KDA_SCAN_INPUT_PLAIN && input_gate != KDA_SCAN_INPUT_COMPLEMENT) return KDA_ERR_INVALID_ARG;
  if (cu && (B != 1 || num_seqs < 1 || !aligned_to(cu, 4))) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

// No rows: the state passes through unchanged.
static kda_status scan_empty(const float* from, float* to, size_t bytes, cudaStream_t stream) {
  if (!to || !bytes || from == to) return KDA_OK;
  return from_cuda(from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, stream)
                        : cudaMemsetAsync(to, 0, bytes, stream));
}

kda_status kda_scan_fwd(const void* x, const void* g, const float* initial_state, const int32_t* cu_seqlens,
                        int num_seqs, void* h, float* final_state, void* checkpoint, int B, int T, int D, int dtype,
                        int prep, int input_gate, void* workspace, size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  kda_status st = scan_flags(B, T, D, cu_seqlens, num_seqs, dtype, prep, input_gate);
  if (st != KDA_OK) return st;
  const int N = cu_seqlens ? num_seqs : 0;
  const size_t nb = (size_t)B * T * D * elem_bytes(dtype), sb = (size_t)(N ? N : B) * D * sizeof(float);
  kda::ScanArgs a{};
  a.x = x, a.g = g, a.s0 = initial_state, a.cu = cu_seqlens, a.out = h, a.sT = final_state;
  a.ckpt = static_cast<uint8_t*>(checkpoint);
  a.B = B, a.T = T, a.D = D, a.N = N, a.dtype = dtype, a.prep = prep, a.complement = input_gate;
  const Range in[] = {{(const char*)x, nb}, {(const char*)g, nb}, {(const char*)initial_state, sb},
                      {(const char*)cu_seqlens, (size_t)(N + 1) * 4}};
  const Range out[] = {{(const char*)h, nb}, {(const char*)final_state, sb},
                       {(const char*)checkpoint, kda::scan_ckpt_layout((size_t)B * T, D).total}};
  const Range need[] = {in[0], in[1], out[0]};
  st = scan_checks(a, in, 4, out, 3, need, 3, workspace, workspace_bytes);
  if (st != KDA_OK) return st;
  if (B == 0 || T == 0) return scan_empty(initial_state, final_state, sb, stream);
  return from_cuda(kda::launch_scan_fwd(a, workspace, stream));
}

kda_status kda_scan_backward(const void* x, const void* g, const void* h, const float* initial_state,
                             const void* grad_h, const float* grad_final_state, const int32_t* cu_seqlens,
                             int num_seqs, void* grad_x, void* grad_g, float* grad_initial_state, int B, int T, int D,
                             int dtype, int prep, int input_gate, void* workspace, size_t workspace_bytes,
                             void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  kda_status st = scan_flags(B, T, D, cu_seqlens, num_seqs, dtype, prep, input_gate);
  if (st != KDA_OK) return st;
  const int N = cu_seqlens ? num_seqs : 0;
  const size_t nb = (size_t)B * T * D * elem_bytes(dtype), sb = (size_t)(N ? N : B) * D * sizeof(float);
  kda::ScanArgs a{};
  a.x = input_gate == KDA_SCAN_INPUT_COMPLEMENT ? x : nullptr;
  a.g = g, a.h = h, a.dy = grad_h, a.s0 = grad_final_state, a.h0 = initial_state, a.cu = cu_seqlens;
  a.out = grad_x, a.dg = grad_g, a.sT = grad_initial_state;
  a.B = B, a.T = T, a.D = D, a.N = N, a.dtype = dtype, a.prep = prep, a.complement = input_gate;
  const Range in[] = {{(const char*)a.x, nb}, {(const char*)g, nb}, {(const char*)h, nb}, {(const char*)grad_h, nb},
                      {(const char*)initial_state, sb}, {(const char*)grad_final_state, sb},
                      {(const char*)cu_seqlens, (size_t)(N + 1) * 4}};
  const Range out[] = {{(const char*)grad_x, nb}, {(const char*)grad_g, nb}, {(const char*)grad_initial_state, sb}};
  const Range need[] = {in[1], in[2], in[3], out[0], out[1],
                        {(const char*)a.x, input_gate == KDA_SCAN_INPUT_COMPLEMENT ? nb : 0}};
  st = scan_checks(a, in, 7, out, 3, need, 6, workspace, workspace_bytes);
  if (st != KDA_OK) return st;
  if (B == 0 || T == 0) return scan_empty(grad_final_state, grad_initial_state, sb, stream);
  return from_cuda(kda::launch_scan_bwd(a, workspace, stream));
}

kda_status kda_scan_backward_ckpt(const void* checkpoint, const void* grad_h, const float* grad_final_state,
                                  const int32_t* cu_seqlens, int num_seqs, void* grad_x, void* grad_g,
                                  float* grad_initial_state, int B, int T, int D, int dtype, int prep, int input_gate,
                                  void* workspace, size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  kda_status st = scan_flags(B, T, D, cu_seqlens, num_seqs, dtype, prep, input_gate);
  if (st != KDA_OK) return st;
  const int N = cu_seqlens ? num_seqs : 0;
  const size_t nb = (size_t)B * T * D * elem_bytes(dtype), sb = (size_t)(N ? N : B) * D * sizeof(float);
  kda::ScanArgs a{};
  a.dy = grad_h, a.s0 = grad_final_state, a.cu = cu_seqlens, a.out = grad_x, a.dg = grad_g, a.sT = grad_initial_state;
  a.ckpt = static_cast<uint8_t*>(const_cast<void*>(checkpoint));
  a.B = B, a.T = T, a.D = D, a.N = N, a.dtype = dtype, a.prep = prep, a.complement = input_gate;
  const Range in[] = {{(const char*)checkpoint, kda::scan_ckpt_layout((size_t)B * T, D).total},
                      {(const char*)grad_h, nb}, {(const char*)grad_final_state, sb},
                      {(const char*)cu_seqlens, (size_t)(N + 1) * 4}};
  const Range out[] = {{(const char*)grad_x, nb}, {(const char*)grad_g, nb}, {(const char*)grad_initial_state, sb}};
  const Range need[] = {in[0], in[1], out[0], out[1]};
  st = scan_checks(a, in, 4, out, 3, need, 4, workspace, workspace_bytes);
  if (st != KDA_OK) return st;
  if (B == 0 || T == 0) return scan_empty(grad_final_state, grad_initial_state, sb, stream);
  return from_cuda(kda::launch_scan_bwd(a, workspace, stream));
}

kda_status kda_scan_step(const void* x, const void* g, const float* state, float* out_state, void* h, int N, int D,
                         int dtype, int prep, int input_gate, void* stream_) {
  const kda_status st = scan_flags(N, 1, D, nullptr, 0, dtype, prep, input_gate);
  if (st != KDA_OK) return st;
  if (N == 0) return KDA_OK;
  const size_t n = (size_t)N * D, nb = n * elem_bytes(dtype);
  const Range in[] = {{(const char*)x, nb}, {(const char*)g, nb}, {(const char*)state, n * 4}};
  const Range out[] = {{(const char*)out_state, n * 4}, {(const char*)h, nb}};
  for (Range r : in)
    if (!r.lo || !aligned16(r.lo)) return KDA_ERR_INVALID_ARG;
  for (Range r : out) {
    if (!r.lo || !aligned16(r.lo)) return KDA_ERR_INVALID_ARG;
    for (Range q : in)
      if (!(r.lo == (const char*)out_state && q.lo == (const char*)state && out_state == state) && overlaps(r, q))
        return KDA_ERR_INVALID_ARG;
  }
  if (overlaps(out[0], out[1])) return KDA_ERR_INVALID_ARG;
  return from_cuda(kda::launch_scan_step(x, g, state, out_state, h, n, dtype, prep, input_gate,
                                         static_cast<cudaStream_t>(stream_)));
}

}  // extern "C"
