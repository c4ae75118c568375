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

// As launch_after, the arguments taken from where they are (they are 20 KB).
template <class A>
cudaError_t launch_args(void (*kernel)(const A), unsigned grid, unsigned block, int shared, int cluster, const A& a,
                        cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = (size_t)shared;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void* args[1] = {const_cast<A*>(&a)};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args);
}

template <class D, int Stage, int Act> cudaError_t launch(const MmaArgs& a, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};
  const auto kernel = ffn_mma_kernel<D, Stage, Act>;
  const cudaError_t e = opt_in(kernel, mma_shared(Stage), &opted);
  if (e != cudaSuccess) return e;
  const int64_t pairs = a.tiles < sms / 2 ? a.tiles : sms / 2;
  return launch_args<MmaArgs>(kernel, (unsigned)(2 * pairs), kMmaThreads, mma_shared(Stage), 2, a, st);
}

template <class D, int Stage, int Act, int Ranks> cudaError_t launch_few(const FewArgs<Ranks>& a, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};
  const auto kernel = ffn_few_kernel<D, Stage, Act, Ranks>;
  const cudaError_t e = opt_in(kernel, kFewRingAlone + 1024, &opted);
  if (e != cudaSuccess) return e;
  return launch_args<FewArgs<Ranks>>(kernel, (unsigned)(a.tiles * a.split), kFewThreads, a.ring + 1024, a.split, a, st);
}

template <int Ranks> cudaError_t few_by_stage(FfnStage stage, const FewArgs<Ranks>& a, cudaStream_t st) {
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

}  // namespace

template <> cudaError_t launch_ffn_few<RA_INST_DTYPE>(FfnStage stage, const FewArgs<kFewRanks>& a, cudaStream_t st) {
  return few_by_stage(stage, a, st);
}
template <> cudaError_t launch_ffn_few<RA_INST_DTYPE>(FfnStage stage, const FewArgs<kMaxRanks>& a, cudaStream_t st) {
  return few_by_stage(stage, a, st);
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
