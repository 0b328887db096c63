// Check of the corrected quotients (quant.cuh) of fp32 values against CUDA's correctly rounded
// division, comparing e4m3 codes: turned keys are fp32, and so are their scales.
//
// A code can differ from the IEEE quotient's only where the two quotients lie on different sides
// of a border between two codes.  Both are within one unit in the last place of x / s, and neither
// depends on the exponents of x and s while nothing underflows.  So every mantissa of s, every
// mantissa that a border has (1 + (2 i + 1) / 16 between normal codes, (1 + 2 i) 2^-10 between
// subnormal ones) and the nine fp32 values of x around border * s are all there is: 2^23 * 16 * 9
// pairs, taken at exponents from the smallest scale that the quotients are used for (2^-90) to
// the largest (2^118), with the border's exponent from the smallest code's to the largest's.
// Prints the pairs checked and the mismatches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>

#include "quant.cuh"

__global__ void check(int s_exp, int q_exp, unsigned long long* bad, unsigned long long* first) {
  const long long total = 16LL << 23;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int b = (int)(i & 15);
    const float s = ldexpf(__uint_as_float(0x3F800000u | (uint32_t)(i >> 4)), s_exp);
    const float rs = __frcp_rn(s);
    // borders of normal codes at 2^q_exp; those of subnormal codes are (1 + 2 i) 2^-10
    const float m = b < 8 ? ldexpf(1.0f + (2 * b + 1) / 16.0f, q_exp)
                          : ldexpf((float)(2 * (b - 8) + 1), -10);
    const uint32_t x0 = __float_as_uint(m * s);
    for (int k = -4; k <= 4; ++k) {
      const float x = __uint_as_float(x0 + k);
      const uint32_t ref = kvfp8::e4m3x2(__fdiv_rn(x, s), __fdiv_rn(-x, s));
      const uint32_t got = kvfp8::e4m3x2(kvfp8::div_by_scale(x, s, rs), kvfp8::div_by_scale(-x, s, rs));
      const uint32_t fresh = kvfp8::e4m3x2(kvfp8::div_fresh(x, s, rs), kvfp8::div_fresh(-x, s, rs));
      if (ref != got || ref != fresh) {
        atomicAdd(bad, 1ull);
        atomicMin(first, (unsigned long long)i);
      }
    }
  }
}

int main() {
  unsigned long long *d_bad, *d_first, h_bad = 0, h_first = ~0ull;
  if (cudaMalloc(&d_bad, 8) != cudaSuccess || cudaMalloc(&d_first, 8) != cudaSuccess) return 2;
  cudaMemset(d_bad, 0, 8);
  cudaMemcpy(d_first, &h_first, 8, cudaMemcpyHostToDevice);
  const int s_exps[] = {-90, -89, -60, -7, 0, 20, 117, 118}, q_exps[] = {-6, -3, 0, 7};
  long long pairs = 0;
  for (int s : s_exps)
    for (int q : q_exps) {
      check<<<152 * 8, 256>>>(s, q, d_bad, d_first);
      pairs += (16LL << 23) * 9;
    }
  if (cudaDeviceSynchronize() != cudaSuccess) {
    printf("cuda error\n");
    return 2;
  }
  cudaMemcpy(&h_bad, d_bad, 8, cudaMemcpyDeviceToHost);
  cudaMemcpy(&h_first, d_first, 8, cudaMemcpyDeviceToHost);
  printf("pairs=%lld mismatches=%llu first=%llu\n", pairs, h_bad, h_first);
  return h_bad ? 1 : 0;
}
