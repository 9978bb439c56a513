// Product of two microscaled 4-bit matrices (qmm_matmul_mx, include/qmm.h) on
// the block-scaled tensor cores.
//
// The weights are the 128-row operand and the activations the narrow one, so a
// call of a few rows pads the activations to 16 only, and a thread of the
// epilogue, which owns one of the 128 accumulator lanes, writes one output
// column: a warp's store covers 32 consecutive columns of a row of Y.
//
// One CTA computes a tile of 128 columns x BN rows over K, or, where there are
// few tiles, a cluster of C CTAs a share of K each, added in rank order through
// distributed shared memory.  Warp 0 copies code tiles (256 codes = 128 bytes a
// row, TMA with the 128-byte swizzle), warps 2..5 the scale bytes, and one
// thread of warp 1 issues, per stage, the copies of the scales into tensor
// memory and four MMAs of 64 codes each.  The scale bytes come from the
// canonical [rows, K/g] layout; a stage holds them as the tensor memory copy
// wants them: per 4 bytes of K (64 codes of nvfp4, 128 of mxfp4) and 128 rows
// 512 bytes, row r's at (r mod 32) * 16 + (r / 32) * 4.
//
// Arithmetic: codes and scales are exact, their products too; the accumulator
// is fp32.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "../../include/qmm.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kTileN = 128;   // columns of Y (rows of W) of a tile: the MMA's M
constexpr int kTileK = 256;   // codes of a stage: 128 bytes a row
constexpr int kGemmThreads = 192;
constexpr int kCodesW = kTileN * kTileK / 2;  // bytes of a stage's weight codes

struct MxMatmulArgs {
  const uint8_t* xs;
  const uint8_t* ws;
  void* Y;
  int M, N, K, out_f32;
  int BN;       // rows of Y of a tile: the MMA's N, a multiple of 16, at most 256
  int tiles_m;  // tiles along M
  int ktiles;   // stages of K
  int split;    // CTAs of a cluster
  int stages;
  int pitch;    // scale bytes of a row
  int words;    // scale bytes can be copied 4 at a time
  uint32_t tmem_cols;
};

// Shared-memory layout (offsets from a 1024-byte aligned start).
struct GemmSmem {
  int x, sfw, sfx, stage;  // within a stage: weight codes, activation codes, scales
  int bars, total;
  __host__ __device__ GemmSmem(int BN, int stages, int sf_words) {
    x = kCodesW;
    sfw = x + ((BN * (kTileK / 2) + 1023) & ~1023);
    sfx = sfw + 512 * sf_words;
    stage = (sfx + ((BN + 127) / 128) * 512 * sf_words + 1023) & ~1023;
    bars = stages * stage;
    total = bars + (2 * stages + 1) * 8 + 16;
  }
};

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t stride_bytes, uint32_t layout) {
  // start address, leading offset (unused: one swizzle atom / one core matrix
  // wide), stride between 8-row groups, version 1, swizzle mode
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (1ull << 16) | (static_cast<uint64_t>(stride_bytes >> 4) << 32) |
         (1ull << 46) | (static_cast<uint64_t>(layout) << 61);
}
constexpr uint32_t kSwizzle128 = 2, kSwizzleNone = 0;

__device__ __forceinline__ void tmem_copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
template <bool NV>
__device__ __forceinline__ void mma_block_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                 bool accumulate) {
  if constexpr (NV) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(accumulate)) : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(accumulate)) : "memory");
  }
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 4 scale bytes of row `row` from byte `at` on; those past the row's end, and
// rows past the matrix, are 0 (their codes are 0 too).
__device__ __forceinline__ uint32_t scale_bytes(const uint8_t* s, int64_t row, int rows, int pitch, int at) {
  uint32_t w = 0;
  if (row < rows)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i < pitch) w |= static_cast<uint32_t>(s[row * pitch + at + i]) << (8 * i);
  return w;
}

template <bool NV>
__global__ void __launch_bounds__(kGemmThreads, 1)
mx_matmul_kernel(const MxMatmulArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap) {
  constexpr int SFW = NV ? 4 : 2;  // 4-byte scale words of a row in a stage
  extern __shared__ __align__(128) unsigned char smem_raw[];
  unsigned char* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const GemmSmem L(a.BN, a.stages, SFW);
  const uint32_t full = sbase + L.bars, empty = full + a.stages * 8, done = empty + a.stages * 8;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L.bars + (2 * a.stages + 1) * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / a.split;
  const int m0 = (tile % a.tiles_m) * a.BN, n0 = (tile / a.tiles_m) * kTileN;
  const int k_begin = a.ktiles * rank / a.split, k_end = a.ktiles * (rank + 1) / a.split;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&wmap);
    prefetch_tmap(&xmap);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full + s * 8, 1 + 128);
      mbar_init(empty + s * 8, 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(a.tmem_cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  // A wait that gave up (a status bit) skips the later ones: wrong results, no hang.
  if (warp == 0) {
    if (lane == 0) {
      bool lost = false;
      const uint32_t bytes = kCodesW + a.BN * (kTileK / 2);
      for (int k = k_begin; k < k_end; ++k) {
        const int it = k - k_begin, s = it % a.stages;
        if (it >= a.stages && !lost) lost = !mbar_wait(empty + s * 8, ((it / a.stages) & 1) ^ 1, kStatusTimeoutEmpty);
        if (lost) break;
        mbar_arrive_expect_tx(full + s * 8, bytes);
        tma_load_2d(sbase + s * L.stage, &wmap, k * (kTileK / 2), n0, full + s * 8);
        tma_load_2d(sbase + s * L.stage + L.x, &xmap, k * (kTileK / 2), m0, full + s * 8);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool lost = false;
      const uint32_t idesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a.BN >> 3) << 17) | (NV ? 0u : 1u << 23) |
                             (static_cast<uint32_t>(kTileN >> 4) << 24);
      const int xb = (a.BN + 127) / 128;  // 128-row blocks of activation scales
      for (int k = k_begin; k < k_end; ++k) {
        const int it = k - k_begin, s = it % a.stages;
        if (!lost) lost = !mbar_wait(full + s * 8, (it / a.stages) & 1, kStatusTimeoutFull);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the scales were written by threads
        const uint32_t base = sbase + s * L.stage;
        const uint32_t sfw = tmem + a.BN + s * (SFW * 4 * (1 + xb)), sfx = sfw + SFW * 4;
#pragma unroll
        for (int w = 0; w < SFW; ++w) {
          tmem_copy_scales(sfw + w * 4, smem_desc(base + L.sfw + w * 512, 128, kSwizzleNone));
          for (int b = 0; b < xb; ++b)
            tmem_copy_scales(sfx + (w * xb + b) * 4, smem_desc(base + L.sfx + (w * xb + b) * 512, 128, kSwizzleNone));
        }
        const uint64_t da = smem_desc(base, 1024, kSwizzle128), db = smem_desc(base + L.x, 1024, kSwizzle128);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // nvfp4: a word of scales for 64 codes; mxfp4: its lower, then its upper half
          const int w = NV ? j : j >> 1;
          const uint32_t id = NV ? 0u : (j & 1) * 2u;
          mma_block_scaled<NV>(tmem, da + j * 2, db + j * 2, idesc | (id << 4) | (id << 29), sfw + w * 4, sfx + w * xb * 4,
                               it > 0 || j > 0);
        }
        mma_commit(empty + s * 8);
      }
      mma_commit(done);
    }
  } else {
    // scale bytes of weight row r and of activation rows r, r + 128
    const int r = threadIdx.x - 64;
    const int at_r = (r & 31) * 16 + (r >> 5) * 4;
    bool lost = false;
    const int xb = (a.BN + 127) / 128;
    for (int k = k_begin; k < k_end; ++k) {
      const int it = k - k_begin, s = it % a.stages;
      if (it >= a.stages && !lost) lost = !mbar_wait(empty + s * 8, ((it / a.stages) & 1) ^ 1, kStatusTimeoutEmpty);
      if (lost) break;
      const uint32_t base = sbase + s * L.stage;
      for (int b = 0; b <= xb; ++b) {  // the weights' block, then the activations'
        const bool isx = b > 0;
        const int64_t row = isx ? static_cast<int64_t>(m0) + (b - 1) * 128 + r : static_cast<int64_t>(n0) + r;
        const int rows = isx ? min(a.M, m0 + a.BN) : a.N;
        const uint8_t* src = isx ? a.xs : a.ws;
#pragma unroll
        for (int w = 0; w < SFW; ++w) {
          const uint32_t dst = base + (isx ? L.sfx + (w * xb + b - 1) * 512 : L.sfw + w * 512) + at_r;
          const int at = (k * SFW + w) * 4;
          if (a.words) {
            const bool ok = row < rows && at < a.pitch;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src + (ok ? row * a.pitch + at : 0)),
                         "r"(ok ? 4 : 0) : "memory");
          } else {
            *reinterpret_cast<uint32_t*>(smem + (dst - sbase)) = scale_bytes(src, row, rows, a.pitch, at);
          }
        }
      }
      if (a.words) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full + s * 8) : "memory");
      else mbar_arrive(full + s * 8);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    mbar_wait(done, 0, kStatusTimeoutDrain);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const int q = warp & 3;
    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int n = n0 + q * 32 + lane;
    float* const part = reinterpret_cast<float*>(smem);  // [BN][128], over the stages
    for (int c = 0; c < a.BN; c += 16) {
      uint32_t v[16];
      tmem_load16(v, acc + c);
      tmem_wait_load();
      if (a.split > 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kTileN + q * 32 + lane] = __uint_as_float(v[i]);
      } else if (n < a.N) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (m0 + c + i < a.M) store_y(a.Y, nullptr, static_cast<int64_t>(m0 + c + i) * a.N + n, __uint_as_float(v[i]), a.out_f32);
      }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncwarp();
  __syncthreads();
  __syncwarp();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(a.tmem_cols));
  if (a.split > 1) {
    // the cluster's partial tiles, added in rank order; each CTA writes its share of the rows
    cluster_sync_all();
    const int rows = min(a.BN, a.M - m0);
    const int r0 = rows * rank / a.split, r1 = rows * (rank + 1) / a.split;
    for (int x = threadIdx.x; x < (r1 - r0) * kTileN; x += kGemmThreads) {
      const int row = r0 + x / kTileN, col = x % kTileN;
      if (n0 + col >= a.N) continue;
      const float* at = reinterpret_cast<const float*>(smem) + row * kTileN + col;
      float v = 0.f;
      for (int c = 0; c < a.split; ++c) v += ld_dsmem_f32(at, c);
      store_y(a.Y, nullptr, static_cast<int64_t>(m0 + row) * a.N + n0 + col, v, a.out_f32);
    }
    cluster_sync_all();  // nobody leaves while its partial tile is read
  }
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Code rows as bytes [rows, K/2], boxes of 128 bytes x `box` rows; what lies
// outside reads as zeros.
bool codes_map(CUtensorMap* map, const void* codes, int rows, int K, int box) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t extent[2] = {kTileK / 2, static_cast<cuuint32_t>(box)};
  const cuuint32_t step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, extent, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tile height and cluster size: the cheapest by an estimate in SM cycles.  A
// stage costs its MMAs (four of 128 x BN x 64) or, from HBM, the bytes that the
// SMs' tiles of one wave need; a tile costs a fixed start and end and its
// outputs.
void plan(MxMatmulArgs& a, int sms) {
  double best = 1e300;
  for (int bn : {16, 32, 64, 128, 256}) {
    if (bn > 16 && bn >= 2 * a.M) break;
    const int64_t tiles = static_cast<int64_t>((a.N + kTileN - 1) / kTileN) * ((a.M + bn - 1) / bn);
    for (int c : {1, 2, 4, 8}) {
      if (c > 1 && (c > a.ktiles / 2 || tiles * c > 2 * sms || bn > 128)) break;
      const int per_sm = bn <= 64 ? 2 : 1;
      const double waves = static_cast<double>((tiles * c + sms * per_sm - 1) / (sms * per_sm));
      const double stage = per_sm * std::max(bn * 1.5, 790.0 / ((a.M + bn - 1) / bn));
      const double cost = waves * ((a.ktiles + c - 1) / c * stage + 2500.0 + bn * 8.0 + (c > 1 ? 1500.0 : 0.0));
      if (cost < best) {
        best = cost;
        a.BN = bn;
        a.split = c;
      }
    }
  }
}

template <bool NV>
cudaError_t launch_mx_matmul(MxMatmulArgs a, const void* Xq, const void* Wq, cudaStream_t stream) {
  if (injected_launch_failure()) return cudaErrorLaunchFailure;
  constexpr int SFW = NV ? 4 : 2;
  a.ktiles = (a.K + kTileK - 1) / kTileK;
  a.pitch = a.K / (NV ? 16 : 32);
  a.words = a.pitch % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.ws)) & 3) == 0;
  plan(a, device_sm_count());
  a.tiles_m = (a.M + a.BN - 1) / a.BN;
  const int64_t ctas = static_cast<int64_t>((a.N + kTileN - 1) / kTileN) * a.tiles_m * a.split;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  // Two CTAs an SM up to 64 rows, else one; stages as shared memory and the
  // tensor memory's columns (accumulators, then each stage's scales) allow.
  const int budget = a.BN <= 64 ? 113 * 1024 : 227 * 1024, cols = a.BN <= 64 ? 256 : 512;
  const int sf_cols = SFW * 4 * (1 + (a.BN + 127) / 128);
  a.stages = 1;
  while (a.stages < 8 && GemmSmem(a.BN, a.stages + 1, SFW).total + 1024 <= budget && a.BN + (a.stages + 1) * sf_cols <= cols)
    ++a.stages;
  a.tmem_cols = cols;
  const int smem = GemmSmem(a.BN, a.stages, SFW).total + 1024;
  CUtensorMap wmap, xmap;
  if (!codes_map(&wmap, Wq, a.N, a.K, kTileN) || !codes_map(&xmap, Xq, a.M, a.K, a.BN)) return cudaErrorNotSupported;
  auto kern = mx_matmul_kernel<NV>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, wmap, xmap);
}

}  // namespace

unsigned int read_mx_matmul_status(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_qmm_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear && v != 0) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_qmm_status, &zero, sizeof(zero));
  }
  return v;
}

}  // namespace qmm

extern "C" qmm_status qmm_matmul_mx(const uint32_t* Xq, const uint8_t* x_scales, const uint32_t* Wq,
                                    const uint8_t* w_scales, int M, int N, int K, int format, void* Y, int out_dtype,
                                    void* stream) {
  using namespace qmm;
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return QMM_ERR_SHAPE;
  if (format != QMM_MXFP4 && format != QMM_NVFP4) return QMM_ERR_UNSUPPORTED;
  if (out_dtype != QMM_OUT_BF16 && out_dtype != QMM_OUT_F32) return QMM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return QMM_OK;
  const size_t esize = out_dtype == QMM_OUT_F32 ? 4 : 2;
  if (Y == nullptr) return QMM_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(Y) % esize) return QMM_ERR_ALIGN;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (K == 0)
    return static_cast<qmm_status>(
        finish_call(cudaMemsetAsync(Y, 0, static_cast<size_t>(M) * static_cast<size_t>(N) * esize, st)));
  if (Xq == nullptr || Wq == nullptr || x_scales == nullptr || w_scales == nullptr) return QMM_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(Xq) | reinterpret_cast<uintptr_t>(Wq)) & 15) return QMM_ERR_ALIGN;
  MxMatmulArgs a = {};
  a.xs = x_scales;
  a.ws = w_scales;
  a.Y = Y;
  a.M = M;
  a.N = N;
  a.K = K;
  a.out_f32 = out_dtype == QMM_OUT_F32;
  const cudaError_t e = format == QMM_NVFP4 ? launch_mx_matmul<true>(a, Xq, Wq, st) : launch_mx_matmul<false>(a, Xq, Wq, st);
  return static_cast<qmm_status>(finish_call(e));
}
