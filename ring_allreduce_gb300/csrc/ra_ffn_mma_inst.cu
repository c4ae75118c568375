// ra_ffn_mma_inst.cu -- the tensor cores' products for one type,
// RA_INST_DTYPE (compiled once per type).
#include "ra_ffn_few.cuh"
#include "ra_ffn_mma.cuh"

#include <atomic>

namespace ra {

namespace {

// Each kernel is opted in to its shared memory once a device.
template <class K> cudaError_t opt_in(K kernel, int shared, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

template <class D, int Stage, int Act> cudaError_t launch(const MmaArgs& a, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};
  const auto kernel = ffn_mma_kernel<D, Stage, Act>;
  const cudaError_t e = opt_in(kernel, mma_shared(Stage), &opted);
  if (e != cudaSuccess) return e;
  const int64_t pairs = a.tiles < sms / 2 ? a.tiles : sms / 2;
  return launch_after(kernel, dim3((unsigned)(2 * pairs)), dim3(kMmaThreads), mma_shared(Stage), st, 2, a);
}

template <class D, int Stage, int Act> cudaError_t launch_few(const FewArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};
  const auto kernel = ffn_few_kernel<D, Stage, Act>;
  const cudaError_t e = opt_in(kernel, kFewRingAlone + 1024, &opted);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3((unsigned)(a.tiles * a.split)), dim3(kFewThreads), (size_t)a.ring + 1024, st, a.split, a);
}

}  // namespace

template <> cudaError_t launch_ffn_few<RA_INST_DTYPE>(FfnStage stage, const FewArgs& a, cudaStream_t st) {
  using D = DTypeOf<RA_INST_DTYPE>::type;
  const cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  const bool silu = a.act == RA_SILU;
  switch (stage) {
    case kFfnHidden: return silu ? launch_few<D, kFfnHidden, RA_SILU>(a, st) : launch_few<D, kFfnHidden, RA_GELU>(a, st);
    case kFfnGradHidden:
      return silu ? launch_few<D, kFfnGradHidden, RA_SILU>(a, st) : launch_few<D, kFfnGradHidden, RA_GELU>(a, st);
    default: return launch_few<D, kFfnOut, RA_SILU>(a, st);
  }
}

template <> cudaError_t launch_ffn_mma<RA_INST_DTYPE>(FfnStage stage, const MmaArgs& a, int sms, cudaStream_t st) {
  using D = DTypeOf<RA_INST_DTYPE>::type;
  const cudaError_t e = debug_upload(st);
  if (e != cudaSuccess) return e;
  const bool silu = a.act == RA_SILU;
  switch (stage) {
    case kFfnHidden:
      return silu ? launch<D, kFfnHidden, RA_SILU>(a, sms, st) : launch<D, kFfnHidden, RA_GELU>(a, sms, st);
    case kFfnGradHidden:
      return silu ? launch<D, kFfnGradHidden, RA_SILU>(a, sms, st) : launch<D, kFfnGradHidden, RA_GELU>(a, sms, st);
    case kFfnGradW: return launch<D, kFfnGradW, RA_SILU>(a, sms, st);
    default: return launch<D, kFfnOut, RA_SILU>(a, sms, st);
  }
}

}  // namespace ra
