// Grouped product of e4m3 rows and e4m3 matrices with one fp32 scale per block of 128, on the
// fifth-generation tensor cores (tcgen05 kind::f8f6f4):
//   out[m, n] = sum_kb sx[m, kb] sw[g, n / 128, kb] sum_{k in block kb} cx[m, k] cw[g, n, k]
// for the rows m of group g, accumulated in fp32; rows of no group are written as zeros.
//
// The scales change every 128 of K, so no MMA may sum across a block: the four MMAs (K = 32) of a
// block fill one of several TMEM accumulators, and the promotion warps add it, times its scale, to
// fp32 registers while the MMAs of the next block run.  Rows are the MMA's M (one TMEM lane, one
// thread per row) and the matrix's rows its N, so a thread's scale is one number per block and the
// promotion costs one packed fma per two elements.
// Per CTA (one per SM, persistent over (row tile, column tile) items):
//   warp 0      TMA producer of the matrix tiles (32 KB per stage: 256 / BN chunks of K = 128)
//   warp 1      MMA issuer
//   warp 2      TMA producer of the row tiles (boxes of 16 to kRows rows)
//   warp 3      TMEM allocation
//   warps 4-11  promotion and stores: two warpgroups, half of the tile's columns each
// An accumulator row that belongs to no row of the tile is fed by whatever shared memory holds and
// is never read.  Every mbarrier wait is bounded; on timeout the kernel records
// MOE_ERR_DEVICE_TIMEOUT and winds down.
#include <algorithm>

#include "group_tiles.cuh"
#include "internal.cuh"
#include "tc_common.cuh"
#include "tensor_map.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kWarpTmaB = 0, kWarpMma = 1, kWarpTmaA = 2, kWarpAlloc = 3, kWarpPromote = 4;
constexpr int kChunk = 128;                    // K of a scale block: one 128-byte swizzled row
constexpr int kBStage = 32768;
constexpr uint32_t kSpinLimit = 1u << 24;      // drain loops only
constexpr uint64_t kWaitTimeoutNs = 1000000000ull;

// BN: columns of a tile (MMA N); kRows: rows of a tile at most.
template <int BN, int kRows>
struct Tile {
  static constexpr int kChunks = 256 / BN;                     // K chunks per stage
  static constexpr int kAStage = kChunks * kRows * kChunk;
  static constexpr int kStages = std::min(4, 196608 / (kAStage + kBStage));
  static constexpr int kBufs = std::min(4, 512 / BN);          // TMEM accumulators
  static constexpr int kTmemCols = kBufs * BN;
  static constexpr int kCols = BN / 2;                         // columns per promoting thread
  static constexpr int kBoxes = kRows / 16;
  static constexpr int kActive = kRows / 32 * 2;               // promotion warps with rows
};

template <int kBoxes>
struct Maps {
  CUtensorMap a[kBoxes];         // row codes, a box of 16 (i + 1) rows x kChunks chunks
  CUtensorMap b;                 // matrix codes, kChunks chunks
  CUtensorMap b_one;             // one chunk
  CUtensorMap b_tail;            // the last chunk of a K that is no multiple of 128
};

struct Bars {
  uint64_t full[4], empty[4];           // stage: two arrivals (matrix and rows), one commit
  uint64_t acc_full[4], acc_empty[4];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* tm, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(tm), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(uint64_t v) {
  const float2 f = unpack2(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 32 bytes of one row (32-byte aligned)
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Stores a thread's kCols columns from column n on of its row.  32-byte stores where rows start on
// 32 bytes (measured against two 16-byte stores: the latter send half sectors), else per element.
template <int kCols>
__device__ __forceinline__ void store_row(const BlockFp8Args& a, int64_t row, int n, const uint64_t (&acc)[kCols / 2],
                                          bool vec) {
  if (a.out_fp32) {
    float* dst = static_cast<float*>(a.out) + row * a.N + n;
    if (vec) {
#pragma unroll
      for (int c = 0; c < kCols; c += 8) {
        if (n + c < a.N) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(acc[c / 2 + i]);
            w[2 * i] = __float_as_uint(f.x);
            w[2 * i + 1] = __float_as_uint(f.y);
          }
          store32(dst + c, w);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < kCols; c += 2) {
        const float2 f = unpack2(acc[c / 2]);
        if (n + c < a.N) dst[c] = f.x;
        if (n + c + 1 < a.N) dst[c + 1] = f.y;
      }
    }
  } else {
    uint16_t* dst = static_cast<uint16_t*>(a.out) + row * a.N + n;
    if (vec) {
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        if (n + c < a.N) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = bf16x2(acc[c / 2 + i]);
          store32(dst + c, w);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < kCols; c += 2) {
        const uint32_t h = bf16x2(acc[c / 2]);
        if (n + c < a.N) dst[c] = static_cast<uint16_t>(h);
        if (n + c + 1 < a.N) dst[c + 1] = static_cast<uint16_t>(h >> 16);
      }
    }
  }
}

template <int BN, int kRows>
__global__ void __launch_bounds__(kThreads, 1)
    block_fp8_kernel(const __grid_constant__ Maps<Tile<BN, kRows>::kBoxes> maps, BlockFp8Args a, bool vec) {
  using C = Tile<BN, kRows>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ GroupTiles gt;
  __shared__ Bars sm;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = base;                                // row tiles first: reads past a short tile stay inside
  uint8_t* sB = base + C::kStages * C::kAStage;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NT = (a.N + BN - 1) / BN;
  const int KB = (a.K + kChunk - 1) / kChunk, KF = a.K / kChunk;
  const int KS = (KB + C::kChunks - 1) / C::kChunks;   // stages per item

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sm.full[s], 2);
      mbar_init(&sm.empty[s], 1);
      mbar_init(&sm.acc_full[s], 1);
      mbar_init(&sm.acc_empty[s], C::kActive);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpAlloc) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  build_group_tiles(gt, a.offsets, a.G, a.M, kRows, a.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int64_t items = static_cast<int64_t>(gt.first[a.G + 1]) * NT;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    return mbar_wait_flag(b, parity, &sm.abort_flag, a.status, kWaitTimeoutNs);
  };
  auto warp_wait = [&](uint64_t* b, uint32_t parity) {
    const bool ok = wait(b, parity);
    return __all_sync(0xffffffffu, ok) != 0;
  };

  if (warp < kWarpPromote) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kWarpTmaB || warp == kWarpTmaA) {
      if (lane == 0) {
        uint32_t is = 0;
        bool ok = true;
        for (int64_t item = blockIdx.x; ok && item < items; item += gridDim.x) {
          const RowTile rt = group_tile(gt, a.G, static_cast<int>(item / NT), kRows);
          if (rt.group == a.G) continue;
          const int n0 = static_cast<int>(item % NT) * BN;
          const int n16 = (rt.rows + 15) >> 4;
          for (int s = 0; s < KS; ++s, ++is) {
            const int st = is % C::kStages, kb0 = s * C::kChunks;
            if (!(ok = wait(&sm.empty[st], ((is / C::kStages) & 1) ^ 1))) break;
            if (warp == kWarpTmaA) {
              mbar_expect_tx(&sm.full[st], C::kChunks * n16 * 16 * kChunk);
              tma_load_3d(sA + st * C::kAStage, &maps.a[n16 - 1], 0, rt.row, kb0, &sm.full[st]);
            } else if (kb0 + C::kChunks <= KF) {
              mbar_expect_tx(&sm.full[st], kBStage);
              tma_load_4d(sB + st * kBStage, &maps.b, 0, n0, kb0, rt.group, &sm.full[st]);
            } else {   // the last stage, chunk by chunk
              mbar_expect_tx(&sm.full[st], (KB - kb0) * BN * kChunk);
              for (int kb = kb0; kb < KB; ++kb) {
                uint8_t* dst = sB + st * kBStage + (kb - kb0) * BN * kChunk;
                if (kb < KF) tma_load_4d(dst, &maps.b_one, 0, n0, kb, rt.group, &sm.full[st]);
                else tma_load_3d(dst, &maps.b_tail, kb * kChunk, n0, rt.group, &sm.full[st]);
              }
            }
          }
        }
        if (!ok) {   // let copies already issued land before the CTA winds down (bounded)
          for (int j = 0; j < C::kStages && is > 0; ++j, --is) {
            const uint32_t q = is - 1;
            for (uint32_t i = 0; i < (1u << 16) && !mbar_try(&sm.full[q % C::kStages], (q / C::kStages) & 1); ++i) {
            }
          }
        }
      }
    } else if (warp == kWarpMma) {
      constexpr uint32_t idesc_rows = 128;
      const uint32_t idesc = idesc_f32acc(idesc_rows, BN);
      uint32_t is = 0, ib = 0;
      bool ok = true;
      for (int64_t item = blockIdx.x; ok && item < items; item += gridDim.x) {
        const RowTile rt = group_tile(gt, a.G, static_cast<int>(item / NT), kRows);
        if (rt.group == a.G) continue;
        const int a_chunk = ((rt.rows + 15) & ~15) * kChunk;
        for (int s = 0; ok && s < KS; ++s, ++is) {
          const int st = is % C::kStages;
          if (!(ok = warp_wait(&sm.full[st], (is / C::kStages) & 1))) break;
          const int chunks = min(C::kChunks, KB - s * C::kChunks);
          for (int c = 0; c < chunks; ++c, ++ib) {
            const int buf = ib % C::kBufs;
            if (!(ok = warp_wait(&sm.acc_empty[buf], ((ib / C::kBufs) & 1) ^ 1))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t aa = smem_u32(sA + st * C::kAStage) + c * a_chunk;
              const uint32_t ba = smem_u32(sB + st * kBStage) + c * BN * kChunk;
#pragma unroll
              for (int kk = 0; kk < kChunk / 32; ++kk)
                mma_e4m3(tmem + buf * BN, smem_desc_sw128(aa + kk * 32), smem_desc_sw128(ba + kk * 32), idesc, kk != 0);
              tc_commit(&sm.acc_full[buf]);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (elect_one()) tc_commit(&sm.empty[st]);
          __syncwarp();
        }
      }
      if (elect_one()) {   // every MMA issued completes before TMEM is released (bounded)
        tc_commit(&sm.drain);
        for (uint32_t i = 0; i < kSpinLimit && !mbar_try(&sm.drain, 0); ++i) {
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int q = warp & 3, half = (warp - kWarpPromote) >> 2;
    if (q * 32 < kRows) {
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * C::kCols;
      const int NB = (a.N + 127) / 128, pitch = (KB + 3) & ~3;
      uint32_t ib = 0;
      bool ok = true;
      for (int64_t item = blockIdx.x; ok && item < items; item += gridDim.x) {
        const RowTile rt = group_tile(gt, a.G, static_cast<int>(item / NT), kRows);
        const int n0 = static_cast<int>(item % NT) * BN + half * C::kCols;
        const bool mine = q * 32 + lane < rt.rows;
        const int64_t row = rt.row + (mine ? q * 32 + lane : 0);
        uint64_t acc[C::kCols / 2];
#pragma unroll
        for (int i = 0; i < C::kCols / 2; ++i) acc[i] = 0;
        if (rt.group < a.G) {
          const bool some = q * 32 < rt.rows;             // rows of this warp
          const float4* sx = reinterpret_cast<const float4*>(a.x_scales + row * pitch);
          const float* sw = a.w_scales + (static_cast<int64_t>(rt.group) * NB + min(n0 / 128, NB - 1)) * KB;
          // scales of four blocks at a time, the next four in flight
          float4 x_next = __ldg(sx);
          float w_next[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w_next[i] = i < KB ? __ldg(sw + i) : 0.0f;
          for (int kb0 = 0; ok && kb0 < KB; kb0 += 4) {
            const float sc[4] = {x_next.x * w_next[0], x_next.y * w_next[1], x_next.z * w_next[2], x_next.w * w_next[3]};
            if (kb0 + 4 < KB) {
              x_next = __ldg(sx + kb0 / 4 + 1);
#pragma unroll
              for (int i = 0; i < 4; ++i) w_next[i] = kb0 + 4 + i < KB ? __ldg(sw + kb0 + 4 + i) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (kb0 + i >= KB) break;
              const int buf = ib % C::kBufs;
              if (!(ok = warp_wait(&sm.acc_full[buf], (ib / C::kBufs) & 1))) break;
              ++ib;
              tc_fence_after();
              if (some) {
                const uint64_t s2 = pack2(__float_as_uint(sc[i]), __float_as_uint(sc[i]));
                const uint32_t t = t_lane + buf * BN;
                uint32_t v[2][16];
                TC_LD16(t, v[0]);
#pragma unroll
                for (int c = 0; c < C::kCols; c += 16) {
                  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                  if (c + 16 < C::kCols) TC_LD16(t + c + 16, v[(c / 16 + 1) & 1]);
#pragma unroll
                  for (int j = 0; j < 8; ++j) fma2(acc[c / 2 + j], pack2(v[(c / 16) & 1][2 * j], v[(c / 16) & 1][2 * j + 1]), s2);
                }
              }
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.acc_empty[buf]);
            }
          }
        }
        if (ok && mine && n0 < a.N) store_row<C::kCols>(a, row, n0, acc, vec);
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpAlloc) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols));
  }
}

template <int BN, int kRows>
cudaError_t launch_tile(const BlockFp8Args& a, int n_sm, cudaStream_t st) {
  using C = Tile<BN, kRows>;
  constexpr int smem = 1024 + C::kStages * (C::kAStage + kBStage);
  auto kern = block_fp8_kernel<BN, kRows>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const uint64_t M = a.M, N = a.N, K = a.K, G = a.G, KB = (K + kChunk - 1) / kChunk, KF = K / kChunk;
  Maps<C::kBoxes> maps;
  bool ok = true;
  for (int i = 0; ok && i < C::kBoxes; ++i) {
    const uint64_t dims[3] = {kChunk, M, KB}, strides[2] = {KB * kChunk, kChunk};
    const uint32_t box[3] = {kChunk, static_cast<uint32_t>(16 * (i + 1)), C::kChunks};
    ok = make_tensor_map(&maps.a[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.x_codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (ok && KF > 0) {
    const uint64_t dims[4] = {kChunk, N, KF, G}, strides[3] = {K, kChunk, N * K};
    const uint32_t box[4] = {kChunk, BN, C::kChunks, 1}, one[4] = {kChunk, BN, 1, 1};
    ok = make_tensor_map(&maps.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a.w_codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tensor_map(&maps.b_one, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, a.w_codes, dims, strides, one, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (ok && K % kChunk) {
    const uint64_t dims[3] = {K, N, G}, strides[2] = {K, N * K};
    const uint32_t box[3] = {kChunk, BN, 1};
    ok = make_tensor_map(&maps.b_tail, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.w_codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (!ok) return cudaErrorInvalidValue;
  const bool vec = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && N % (a.out_fp32 ? 8 : 16) == 0;
  // tiles at most: one per full tile of rows and one more per group that has rows
  const int64_t most = (M / kRows + std::min(M, G + 1)) * ((N + BN - 1) / BN);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, n_sm)));
  return launch_pdl(true, kern, dim3(grid), dim3(kThreads), smem, st, maps, a, vec);
}

}  // namespace

cudaError_t launch_block_fp8_matmul(const BlockFp8Args& a, cudaStream_t st) {
  int n_sm = 0;
  cudaError_t e = current_sm_count(&n_sm);
  if (e != cudaSuccess) return e;
  const int64_t large = (a.M / 128 + std::min<int64_t>(a.M, a.G)) * ((a.N + 255) / 256);
  if (a.M <= 16 * static_cast<int64_t>(a.G) || large < n_sm) return launch_tile<64, 32>(a, n_sm, st);
  return launch_tile<256, 128>(a, n_sm, st);
}

}  // namespace moe
