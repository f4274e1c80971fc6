// The bf16 products grouped by expert with ragged sizes: instances and launches of
// the kernel in dg_bf16_kernel.cuh.
#include "dg_bf16_kernel.cuh"

namespace dgk {
namespace {

template <int FORM>
cudaError_t set_up_form() {
  const void* kernels[] = {reinterpret_cast<const void*>(bf16_grouped_kernel<true, 256, FORM, kBfPlain>),
                           reinterpret_cast<const void*>(bf16_grouped_kernel<false, 128, FORM, kBfPlain>),
                           reinterpret_cast<const void*>(bf16_grouped_kernel<false, 64, FORM, kBfPlain>)};
  for (const void* k : kernels) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBfMaxSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int FORM>
cudaError_t launch_form(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode, int num_sms,
                        cudaStream_t stream) {
  const BfPlan f = c.forced.lanes > 0 ? c.forced : bf_plan(c, num_sms);
  return f.pair       ? launch_tiles<true, 256, FORM>(c, encode, f, num_sms, stream)
         : f.bc <= 64 ? launch_tiles<false, 64, FORM>(c, encode, f, num_sms, stream)
                      : launch_tiles<false, 128, FORM>(c, encode, f, num_sms, stream);
}

}  // namespace

// As many CTAs (pairs) as there can be tiles, at most one per SM; with a split
// reduction a cluster for each of them.
long long bf16_grid(const BfCall& c, const BfPlan& f, int num_sms) {
  const long long most = bf_most_tiles(c, f.lanes, f.bc);
  const int width = f.pair ? 2 : 1;
  return std::max(1ll, f.split > 1 ? most : std::min<long long>(most, num_sms / width)) * width * f.split;
}

cudaError_t bf16_set_up() {
  cudaError_t e = set_up_form<kBfNT>();
  if (e == cudaSuccess) e = set_up_form<kBfNN>();
  if (e == cudaSuccess) e = set_up_form<kBfTN>();
  return e;
}

cudaError_t launch_bf16_grouped(const BfCall& c, PFN_cuTensorMapEncodeTiled_v12000 encode,
                                int num_sms, cudaStream_t stream) {
  switch (c.form) {
    case kBfNT: return launch_form<kBfNT>(c, encode, num_sms, stream);
    case kBfNN: return launch_form<kBfNN>(c, encode, num_sms, stream);
    default: return launch_form<kBfTN>(c, encode, num_sms, stream);
  }
}

}  // namespace dgk
