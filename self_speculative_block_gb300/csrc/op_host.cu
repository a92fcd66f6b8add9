// Host helpers of the single-kernel entry points that live in files of their
// own, and the status call of the kernels that report through device words.
#include "../../include/gocr.h"
#include "kernels.cuh"
#include "tc.cuh"

#include <cstdarg>
#include <cstdio>

namespace gocr {

int op_fail(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_lib_error(buf);
  return code;
}

int op_stream_check(cudaStream_t s) {
  // the default streams (null, legacy, per-thread) are the current device's
  if (s == nullptr || s == cudaStreamLegacy || s == cudaStreamPerThread) return GOCR_OK;
  // asking a capturing stream for its device would end the capture; there the
  // launches themselves refuse a foreign stream
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cap) == cudaSuccess && cap != cudaStreamCaptureStatusNone) return GOCR_OK;
  int cur = 0, dev = 0;
  if (cudaGetDevice(&cur) != cudaSuccess || cudaStreamGetDevice(s, &dev) != cudaSuccess) {
    cudaGetLastError();
    return op_fail(GOCR_ECUDA, "cannot read the current or the stream's device");
  }
  if (cur != dev) return op_fail(GOCR_EINVAL, "the stream belongs to another device than the current one");
  return GOCR_OK;
}

int op_launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return op_fail(GOCR_ECUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
  return GOCR_OK;
}

}  // namespace gocr

using namespace gocr;

namespace {

__device__ unsigned g_probe;  // as the operators' counts

// A wait on a barrier that nothing arrives on.
__global__ void wait_probe_kernel(unsigned long long limit) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bar, 1);
    tc::fence_mbar_init();
  }
  __syncthreads();
  if (!tc::mbar_wait_ns(&bar, 0, limit) && threadIdx.x == 0) atomicAdd(&g_probe, 1u);
}

// What a thread has seen of a device's counts.
constexpr int COUNTS = 5, DEVICES = 64;
thread_local unsigned t_seen[DEVICES][COUNTS];

bool capturing(cudaStream_t s) {
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) {
    cudaGetLastError();  // the legacy stream, while another one is being captured
    return true;
  }
  return cap != cudaStreamCaptureStatusNone;
}

}  // namespace

extern "C" int gocr_op_status(void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  if (capturing(s)) return op_fail(GOCR_EINVAL, "a stream that is being captured cannot be waited for");
  if (int rc = op_stream_check(s)) return rc;
  unsigned now[COUNTS] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = linear_ce_gave_up(now, s);
  if (e == cudaSuccess) e = attn_packed_gave_up(now + 1, s);
  if (e == cudaSuccess) e = attn_packed_bwd_gave_up(now + 2, s);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(now + 3, g_probe, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = attn_packed_bwd_unaligned(now + 4, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return op_fail(GOCR_ECUDA, "status read failed: %s", cudaGetErrorString(e));
  }
  if (dev >= DEVICES) return op_fail(GOCR_ECUDA, "device %d: no more than %d are served", dev, DEVICES);
  bool grown[COUNTS];
  for (int i = 0; i < COUNTS; ++i) {
    grown[i] = now[i] != t_seen[dev][i];
    t_seen[dev][i] = now[i];
  }
  if (grown[4]) return op_fail(GOCR_EDEVICE, "a kernel of attention_packed_backward was given unaligned shared memory");
  static const char* const who[4] = {"linear_ce", "attention_packed", "attention_packed_backward", "wait_probe"};
  for (int i = 0; i < 4; ++i)
    if (grown[i]) return op_fail(GOCR_EDEVICE, "a wait inside a kernel of %s gave up", who[i]);
  return GOCR_OK;
}

extern "C" int gocr_op_wait_probe(int microseconds, void* stream) {
  if (microseconds < 1 || microseconds > 1000000) return op_fail(GOCR_EINVAL, "a wait of %d microseconds", microseconds);
  if (int rc = op_stream_check((cudaStream_t)stream)) return rc;
  wait_probe_kernel<<<1, 32, 0, (cudaStream_t)stream>>>(microseconds * 1000ull);
  return op_launched("wait_probe");
}
