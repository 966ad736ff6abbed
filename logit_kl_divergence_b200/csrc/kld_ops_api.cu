// kld_ops_api.cu -- host side of the logit checkpoints' writing and restoring
// and of beam search (include/kld_stats.h): argument checks, the beam handle
// and its workspace. The kernels are in kld_pack.cu and kld_beam.cu.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <new>

#include "kld_host.h"
#include "kld_internal.h"

using kld::cuda_fail;
using kld::DeviceGuard;

struct kld_beam_s {
  int device = 0;
  int sm_count = 0;
  int max_groups = 0, max_beams = 0, max_k = 0, cap = 0;
  void* mem = nullptr;
  float4* sums = nullptr;
  float2* entries = nullptr;
  unsigned* tickets = nullptr;
  uint32_t* flags = nullptr;
  cudaEvent_t done = nullptr;
};

namespace {

bool valid_dtype(kld_dtype_t dt) { return dt == KLD_F32 || dt == KLD_BF16 || dt == KLD_F16; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

kld_status_t check_matrix(const void* x, int64_t N, int64_t V, kld_dtype_t dtype,
                          const kld_packed_t* packed, int device) {
  if (!valid_dtype(dtype)) return KLD_ERR_DTYPE;
  if (!x || !packed || !packed->codes || !packed->heads || device < 0) return KLD_ERR_INVALID_ARG;
  if (N < 1 || V < 1 || V > INT32_MAX || N > INT64_MAX / 4 / (V + KLD_PACK_BLOCK))
    return KLD_ERR_INVALID_ARG;
  if (!aligned(x, static_cast<uintptr_t>(kld::elem_bytes(dtype))) || !aligned(packed->codes, 16) ||
      !aligned(packed->heads, 4))
    return KLD_ERR_INVALID_ARG;
  const int64_t nb = (V + KLD_PACK_BLOCK - 1) / KLD_PACK_BLOCK, bytes = N * V * kld::elem_bytes(dtype);
  if (!kld::apart(x, bytes, packed->codes, N * nb * KLD_PACK_BLOCK) ||
      !kld::apart(x, bytes, packed->heads, 4 * N * nb) ||
      !kld::apart(packed->codes, N * nb * KLD_PACK_BLOCK, packed->heads, 4 * N * nb))
    return KLD_ERR_INVALID_ARG;
  return KLD_OK;
}

// Zeroes device memory before it returns: cudaMemset alone may still be under
// way, and streams that do not wait for the default one would not wait for it.
cudaError_t clear(void* p, size_t bytes) {
  const cudaError_t e = cudaMemset(p, 0, bytes);
  return e != cudaSuccess ? e : cudaStreamSynchronize(nullptr);
}

// The event that kld_beam_status and kld_beam_destroy wait for; not part of
// a captured graph (whose replays the caller waits for).
kld_status_t mark_done(kld_beam_s* h, cudaStream_t s) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  KLD_CUDA(cudaStreamIsCapturing(s, &cap));
  if (cap == cudaStreamCaptureStatusNone) KLD_CUDA(cudaEventRecord(h->done, s));
  return KLD_OK;
}

}  // namespace

extern "C" {

kld_status_t kld_pack_logits(const void* logits, int64_t N, int64_t V, kld_dtype_t dtype,
                             const kld_packed_t* out, int device, void* stream) {
  return kld_pack_logits_masked(logits, N, V, dtype, -INFINITY, out, device, stream);
}

kld_status_t kld_pack_logits_masked(const void* logits, int64_t N, int64_t V, kld_dtype_t dtype,
                                    float mask_at, const kld_packed_t* out, int device,
                                    void* stream) {
  kld_status_t st = check_matrix(logits, N, V, dtype, out, device);
  if (st != KLD_OK) return st;
  if (!(mask_at < INFINITY)) return KLD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = kld::check_device(device, &sms)) != KLD_OK) return st;
  DeviceGuard guard(device);
  if (!guard.ok()) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
  KLD_CUDA(kld::launch_pack(logits, N, V, dtype, mask_at, out->codes, out->heads, sms,
                            static_cast<cudaStream_t>(stream)));
  return KLD_OK;
}

kld_status_t kld_unpack_logits(const kld_packed_t* packed, int64_t N, int64_t V, void* out,
                               kld_dtype_t dtype, int device, void* stream) {
  kld_status_t st = check_matrix(out, N, V, dtype, packed, device);
  if (st != KLD_OK) return st;
  int sms = 0;
  if ((st = kld::check_device(device, &sms)) != KLD_OK) return st;
  DeviceGuard guard(device);
  if (!guard.ok()) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
  KLD_CUDA(kld::launch_unpack(packed->codes, packed->heads, N, V, out, dtype, sms,
                              static_cast<cudaStream_t>(stream)));
  return KLD_OK;
}

kld_status_t kld_beam_create(kld_beam_t* out, int max_groups, int max_beams, int max_k,
                             int device) {
  if (!out) return KLD_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_groups < 1 || max_beams < 1 || max_beams > KLD_BEAM_MAX_BEAMS || max_k < 1 ||
      max_k > KLD_BEAM_MAX_K || device < 0 || max_groups > (1 << 24) / max_beams)
    return KLD_ERR_INVALID_ARG;
  int sms = 0;
  const kld_status_t dev = kld::check_device(device, &sms);
  if (dev != KLD_OK) return dev;
  DeviceGuard guard(device);
  if (!guard.ok()) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
  kld_beam_s* h = new (std::nothrow) kld_beam_s();
  if (!h) return KLD_ERR_OOM;
  h->device = device;
  h->sm_count = sms;
  h->max_groups = max_groups;
  h->max_beams = max_beams;
  h->max_k = max_k;
  // Entries a CTA may leave (a power of two; it leaves about k for every
  // doubling of its tiles); past this it leaves its exact k.
  h->cap = 128;
  while (h->cap < 8 * max_k) h->cap *= 2;
  // One allocation; plan_beam keeps parts * rows within this many parts.
  auto up = [](size_t b) { return (b + 255) & ~static_cast<size_t>(255); };
  const size_t parts = static_cast<size_t>(kld::kBeamSlices) +
                       2 * static_cast<size_t>(max_groups) * static_cast<size_t>(max_beams);
  const size_t sums_b = up(parts * sizeof(float4));
  const size_t entries_b = up(parts * static_cast<size_t>(h->cap) * sizeof(float2));
  const size_t tickets_b = up(static_cast<size_t>(max_groups) * sizeof(unsigned) + sizeof(uint32_t));
  kld_status_t st = KLD_OK;
  cudaError_t err = cudaMalloc(&h->mem, tickets_b + sums_b + entries_b);
  if (err != cudaSuccess) {
    h->mem = nullptr;
    st = cuda_fail(err, "cudaMalloc(beam workspace)");
  } else if ((err = clear(h->mem, tickets_b)) != cudaSuccess) {
    st = cuda_fail(err, "cudaMemset");
  } else if ((err = cudaEventCreateWithFlags(&h->done, cudaEventDisableTiming)) != cudaSuccess) {
    h->done = nullptr;
    st = cuda_fail(err, "cudaEventCreate");
  }
  if (st != KLD_OK) {
    kld_beam_destroy(h);
    return st;
  }
  char* m = static_cast<char*>(h->mem);
  h->tickets = reinterpret_cast<unsigned*>(m);
  h->flags = h->tickets + max_groups;
  h->sums = reinterpret_cast<float4*>(m + tickets_b);
  h->entries = reinterpret_cast<float2*>(m + tickets_b + sums_b);
  *out = h;
  return KLD_OK;
}

void kld_beam_destroy(kld_beam_t h) {
  if (!h) return;
  DeviceGuard guard(h->device);
  if (h->done) {
    cudaEventSynchronize(h->done);
    cudaEventDestroy(h->done);
  }
  if (h->mem) cudaFree(h->mem);
  delete h;
}

kld_status_t kld_beam_select(kld_beam_t h, const void* logits, int64_t ld, kld_dtype_t dtype,
                             const float* scores, const uint8_t* finished, int32_t eos, int groups,
                             int beams, int64_t V, int k, float* scores_out, int32_t* tokens_out,
                             int32_t* parents_out, void* stream) {
  if (!h) return KLD_ERR_INVALID_ARG;
  if (!valid_dtype(dtype)) return KLD_ERR_DTYPE;
  if (!logits || !scores || !scores_out || !tokens_out || !parents_out) return KLD_ERR_INVALID_ARG;
  if (groups < 1 || groups > h->max_groups || beams < 1 || beams > h->max_beams || k < 1 ||
      k > h->max_k || V < 1 || V > INT32_MAX || ld < V ||
      static_cast<int64_t>(beams) * V > static_cast<int64_t>(UINT32_MAX))
    return KLD_ERR_INVALID_ARG;
  if (ld > INT64_MAX / 4 / (static_cast<int64_t>(groups) * beams)) return KLD_ERR_INVALID_ARG;
  if (finished && (eos < 0 || eos >= V)) return KLD_ERR_INVALID_ARG;
  if (!aligned(logits, static_cast<uintptr_t>(kld::elem_bytes(dtype))) || !aligned(scores, 4) ||
      !aligned(scores_out, 4) || !aligned(tokens_out, 4) || !aligned(parents_out, 4))
    return KLD_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(groups) * beams, places = 4 * static_cast<int64_t>(groups) * k;
  const int64_t read = ((rows - 1) * ld + V) * kld::elem_bytes(dtype);
  const void* outs[3] = {scores_out, tokens_out, parents_out};
  for (int i = 0; i < 3; ++i) {
    if (!kld::apart(outs[i], places, logits, read) || !kld::apart(outs[i], places, scores, 4 * rows) ||
        !kld::apart(outs[i], places, finished, rows) ||
        !kld::apart(outs[i], places, outs[(i + 1) % 3], places))
      return KLD_ERR_INVALID_ARG;
  }
  DeviceGuard guard(h->device);
  if (!guard.ok()) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
  kld::BeamSelect b;
  b.logits = logits;
  b.ld = ld;
  b.dtype = dtype;
  b.scores = scores;
  b.finished = finished;
  b.eos = eos;
  b.groups = groups;
  b.beams = beams;
  b.k = k;
  b.cap = h->cap;
  b.V = V;
  b.sums = h->sums;
  b.entries = h->entries;
  b.tickets = h->tickets;
  b.flags = h->flags;
  b.out_scores = scores_out;
  b.out_tokens = tokens_out;
  b.out_parents = parents_out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KLD_CUDA(kld::launch_beam_select(b, h->sm_count, s));
  return mark_done(h, s);
}

kld_status_t kld_beam_reorder(kld_beam_t h, const kld_state_t* states, int n,
                              const int32_t* parents, const int32_t* lengths, int groups,
                              int beams, void* stream) {
  if (!h || n < 0 || (n > 0 && !states) || !parents) return KLD_ERR_INVALID_ARG;
  if (groups < 1 || groups > h->max_groups || beams < 1 || beams > h->max_beams)
    return KLD_ERR_INVALID_ARG;
  if (!aligned(parents, 4) || !aligned(lengths, 4)) return KLD_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const kld_state_t& t = states[i];
    if (t.outer < 0 || t.positions < 0 || t.position_bytes < 0 || t.row_stride < 0 ||
        t.outer_stride < 0 || t.outer > INT32_MAX)
      return KLD_ERR_INVALID_ARG;
    if (t.outer == 0 || t.positions == 0 || t.position_bytes == 0) continue;
    if (!t.data || t.positions > INT64_MAX / t.position_bytes) return KLD_ERR_INVALID_ARG;
    // Runs of a row, and rows, may not overlap.
    const int64_t run = t.positions * t.position_bytes;
    if (t.outer > 1 && t.outer_stride < run) return KLD_ERR_INVALID_ARG;
    if (t.outer > 1 && t.outer_stride > (INT64_MAX - run) / t.outer) return KLD_ERR_INVALID_ARG;
    const int64_t row = t.outer > 1 ? (t.outer - 1) * t.outer_stride + run : run;
    if (static_cast<int64_t>(groups) * beams > 1 && t.row_stride < row) {
      // Rows may also interleave inside the runs' spacing (rows between runs).
      const bool between = t.outer > 1 && t.row_stride >= run &&
                           static_cast<int64_t>(groups) * beams * t.row_stride <= t.outer_stride;
      if (!between) return KLD_ERR_INVALID_ARG;
    }
  }
  DeviceGuard guard(h->device);
  if (!guard.ok()) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = kld::launch_beam_reorder(states, n, parents, lengths, groups, beams, h->flags, s);
  if (e == cudaErrorInvalidConfiguration) return KLD_ERR_INVALID_ARG;  // more runs than a grid holds
  KLD_CUDA(e);
  return mark_done(h, s);
}

kld_status_t kld_beam_status(kld_beam_t h, uint32_t* flags) {
  if (!h || !flags) return KLD_ERR_INVALID_ARG;
  DeviceGuard guard(h->device);
  if (!guard.ok()) return cuda_fail(cudaGetLastError(), "cudaSetDevice");
  KLD_CUDA(cudaEventSynchronize(h->done));
  KLD_CUDA(cudaMemcpy(flags, h->flags, sizeof(uint32_t), cudaMemcpyDeviceToHost));
  KLD_CUDA(clear(h->flags, sizeof(uint32_t)));
  return KLD_OK;
}

}  // extern "C"
