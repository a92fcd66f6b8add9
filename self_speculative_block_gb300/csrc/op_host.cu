// Host helpers of the single-kernel entry points that live in files of their
// own, and the status call of the kernels that report through device words.
#include "../../include/gocr.h"
#include "kernels.cuh"

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

extern "C" int gocr_op_status(void* stream) {
  if (int rc = op_stream_check((cudaStream_t)stream)) return rc;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  int ce = 0, af = 0, ab = 0;
  if (e == cudaSuccess) e = take_linear_ce_error(&ce);
  if (e == cudaSuccess) e = take_attn_packed_error(&af);
  if (e == cudaSuccess) e = take_attn_packed_bwd_error(&ab);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return op_fail(GOCR_ECUDA, "status read failed: %s", cudaGetErrorString(e));
  }
  if (ce || af || ab)
    return op_fail(GOCR_EDEVICE, "a wait inside a kernel of %s gave up",
                   ce ? "linear_ce" : (af ? "attention_packed" : "attention_packed_backward"));
  return GOCR_OK;
}
