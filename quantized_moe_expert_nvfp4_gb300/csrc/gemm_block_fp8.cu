// Grouped product of e4m3 rows and e4m3 matrices with one fp32 scale per block of 128:
//   out[m, n] = sum_kb sx[m, kb] sw[g, n / 128, kb] sum_{k in block kb} cx[m, k] cw[g, n, k]
// for the rows m of group g, accumulated in fp32; rows of no group are written as zeros.
#include <algorithm>

#include "group_tiles.cuh"
#include "internal.cuh"

namespace moe {
namespace {

constexpr int kTM = 32, kTN = 64, kTK = 32;

__global__ void __launch_bounds__(256) block_fp8_simt_kernel(BlockFp8Args a) {
  __shared__ GroupTiles gt;
  __shared__ float sx[kTM][kTK + 1], sw[kTN][kTK + 1];
  pdl_wait();
  build_group_tiles(gt, a.offsets, a.G, a.M, kTM, a.status);
  const int NT = (a.N + kTN - 1) / kTN;
  const int64_t items = static_cast<int64_t>(gt.first[a.G + 1]) * NT;
  const int KB = (a.K + 127) / 128, pitch = (KB + 3) & ~3, NB = (a.N + 127) / 128;
  const int c = threadIdx.x & 63, r0 = threadIdx.x >> 6;   // column c, rows r0, r0 + 4, ...
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const RowTile rt = group_tile(gt, a.G, static_cast<int>(item / NT), kTM);
    const int n0 = static_cast<int>(item % NT) * kTN;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int kb = 0; kb < KB && rt.group < a.G; ++kb) {
      float part[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) part[i] = 0.0f;
      for (int k0 = kb * 128; k0 < kb * 128 + 128; k0 += kTK) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTM * kTK; i += 256) {
          const int r = i / kTK, k = k0 + i % kTK;
          sx[r][i % kTK] = r < rt.rows && k < a.K ? e4m3_to_f32(a.x_codes[static_cast<int64_t>(rt.row + r) * KB * 128 + k]) : 0.0f;
        }
        for (int i = threadIdx.x; i < kTN * kTK; i += 256) {
          const int n = n0 + i / kTK, k = k0 + i % kTK;
          sw[i / kTK][i % kTK] =
              n < a.N && k < a.K ? e4m3_to_f32(a.w_codes[(static_cast<int64_t>(rt.group) * a.N + n) * a.K + k]) : 0.0f;
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < kTK; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) part[i] = fmaf(sx[r0 + 4 * i][k], sw[c][k], part[i]);
      }
      const int nb = min(n0 + c, a.N - 1) / 128;
      const float s = __ldg(a.w_scales + (static_cast<int64_t>(rt.group) * NB + nb) * KB + kb);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r0 + 4 * i < rt.rows)
          acc[i] = fmaf(__ldg(a.x_scales + static_cast<int64_t>(rt.row + r0 + 4 * i) * pitch + kb) * s, part[i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + 4 * i >= rt.rows || n0 + c >= a.N) continue;
      const int64_t o = static_cast<int64_t>(rt.row + r0 + 4 * i) * a.N + n0 + c;
      if (a.out_fp32) static_cast<float*>(a.out)[o] = acc[i];
      else static_cast<uint16_t*>(a.out)[o] = f32_to_bf16_bits(acc[i]);
    }
  }
}

}  // namespace

cudaError_t launch_block_fp8_matmul(const BlockFp8Args& a, cudaStream_t st) {
  int n_sm = 0;
  cudaError_t e = current_sm_count(&n_sm);
  if (e != cudaSuccess) return e;
  return launch_pdl(true, block_fp8_simt_kernel, dim3(4 * n_sm), dim3(256), 0, st, a);
}

}  // namespace moe
