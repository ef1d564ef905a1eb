// Host calls that compare device functions of csrc/adamw.cu with CUDA's own over
// a whole binade (tests/test_gpu_adamw_math.py).
#include "../../moe_expert_layer_ep_gb300/csrc/adamw.cu"

namespace {

// x: every number of the binade 2^e.  out[0]: roots that differ from the rounded
// one; out[1]: the most by which one does, in units in the last place.
__global__ void compare_roots(int e, unsigned long long* out) {
  const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
  const float x = __uint_as_float((static_cast<uint32_t>(e + 127) << 23) | (i & 0x7FFFFFu));
  const int ulps = abs(__float_as_int(moe::sqrt_newton(x)) - __float_as_int(__fsqrt_rn(x)));
  if (ulps) {
    atomicAdd(&out[0], 1ull);
    atomicMax(&out[1], static_cast<unsigned long long>(ulps));
  }
}

// The same of the reciprocal: ulps from the rounded quotient.
__global__ void compare_reciprocals(int e, unsigned long long* out) {
  const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
  const float x = __uint_as_float((static_cast<uint32_t>(e + 127) << 23) | (i & 0x7FFFFFu));
  const int ulps = abs(__float_as_int(moe::rcp_fast(x)) - __float_as_int(__fdiv_rn(1.0f, x)));
  if (ulps) {
    atomicAdd(&out[0], 1ull);
    atomicMax(&out[1], static_cast<unsigned long long>(ulps));
  }
}

}  // namespace

// out: two numbers in device memory, zeros; what: 0 roots, 1 reciprocals.
extern "C" int adamw_compare(int what, int e, unsigned long long* out) {
  if (what)
    compare_reciprocals<<<(1 << 23) / 256, 256>>>(e, out);
  else
    compare_roots<<<(1 << 23) / 256, 256>>>(e, out);
  return static_cast<int>(cudaDeviceSynchronize());
}
