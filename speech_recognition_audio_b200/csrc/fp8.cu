// 8-bit floating point with a power-of-two scale per block of 128: the
// quantiser and the dense layer on quantised operands.
//
//   quantise  s = the smallest integer with amax <= 448 * 2^s over the block
//             (448 is e4m3's largest value), code = e4m3(x * 2^-s), rounded
//             to nearest, ties to even.  The product with a power of two is
//             exact, so the code's rounding is the only one.
//   linear    acc[m, n] = sum over k of 2^(sx[m, k/128] + sw[n/128, k/128])
//             xc[m, k] wc[n, k], on tcgen05 kind::mxf8f6f4: the tensor core
//             applies the E8M0 scales to each 32-wide step itself and
//             accumulates in fp32, so no partial sum leaves tensor memory.
#include <cuda_fp8.h>

#include "gemm.cuh"
#include "kernels.h"

namespace asr {

namespace {

// ------------------------------------------------------------------ quantise

constexpr int QZ_THREADS = 256;
constexpr int QZ_UNROLL = 4;  // blocks of 128 in flight per half-warp

// Eight consecutive elements as fp32 (16-byte loads; the pointer is aligned).
template <int DT>
__device__ __forceinline__ void load8(const void* x, long long i, float* v) {
  if constexpr (DT == SPLICE_F32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + i);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + i));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == SPLICE_BF16) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  }
}

// Largest finite magnitude of the eight values as its bit pattern (which
// orders like the value), and whether any of them is not finite.
__device__ __forceinline__ unsigned int amax8(const float* v, bool& special) {
  unsigned int m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const unsigned int b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    special |= b >= 0x7F800000u;
    m = max(m, b >= 0x7F800000u ? 0u : b);
  }
  return m;
}

// Exponent s of the block's scale from the bits of its largest magnitude:
// amax = f 2^e with f in [1, 2) and 448 = 1.75 * 2^8, so s = e - 8, or e - 7
// where f > 1.75; at least -127 (E8M0's smallest), 0 for a block of zeros.
__device__ __forceinline__ int scale_exp(unsigned int amax_bits) {
  if (amax_bits == 0) return 0;
  const int e = static_cast<int>(amax_bits >> 23) - 127;
  return max(e - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), -127);
}

// The eight codes of v * 2^-s.  Infinities become NaN codes (e4m3 has no
// infinity, and the conversion would saturate them to a finite value).
__device__ __forceinline__ uint2 codes8(const float* v, int s, bool special) {
  const float up = __uint_as_float(static_cast<unsigned int>(127 - s) << 23);  // s in [-127, 120]
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * j] * up, v[2 * j + 1] * up), __NV_SATFINITE, __NV_E4M3);
    if (special) {
      if (!(fabsf(v[2 * j]) < INFINITY)) h[j] = (h[j] & 0xFF00u) | 0x7Fu;
      if (!(fabsf(v[2 * j + 1]) < INFINITY)) h[j] = (h[j] & 0x00FFu) | 0x7F00u;
    }
  }
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

}  // namespace

// One scale per row and 128 columns.  Sixteen lanes share a block (eight
// elements each: whole 16-byte loads and 8-byte code stores, a 128-byte
// segment per block), four blocks in flight per half-warp.
template <int DT>
__global__ void __launch_bounds__(QZ_THREADS) quantize_rows_kernel(const void* __restrict__ x, long long ldx, int K,
                                                                   int KB, unsigned int units,
                                                                   uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int l16 = threadIdx.x & 15;
  const unsigned int first = blockIdx.x * (QZ_THREADS / 16 * QZ_UNROLL) + (threadIdx.x >> 4);
  float v[QZ_UNROLL][8];
  unsigned int row[QZ_UNROLL];
  int kb[QZ_UNROLL];
#pragma unroll
  for (int i = 0; i < QZ_UNROLL; ++i) {
    const unsigned int u = first + i * (QZ_THREADS / 16);
    row[i] = u / static_cast<unsigned int>(KB);
    kb[i] = static_cast<int>(u - row[i] * KB);
    const int k = kb[i] * 128 + 8 * l16;
    if (u < units && k < K) {
      load8<DT>(x, row[i] * ldx + k, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < QZ_UNROLL; ++i) {
    const unsigned int u = first + i * (QZ_THREADS / 16);
    bool special = false;
    unsigned int m = amax8(v[i], special);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int s = scale_exp(m);
    const int k = kb[i] * 128 + 8 * l16;
    if (u < units) {
      if (k < K) *reinterpret_cast<uint2*>(codes + (long long)row[i] * K + k) = codes8(v[i], s, special);
      if (l16 == 0) scales[u] = static_cast<uint8_t>(s + 127);
    }
  }
}

// One scale per 128 x 128 block (weights): one thread block each, the 128
// rows in eight passes of sixteen, held in registers between the maximum and
// the conversion.
template <int DT>
__global__ void __launch_bounds__(QZ_THREADS) quantize_blocks_kernel(const void* __restrict__ x, long long ldx,
                                                                     long long M, int K, int KB,
                                                                     uint8_t* __restrict__ codes,
                                                                     uint8_t* __restrict__ scales) {
  __shared__ unsigned int wmax[QZ_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  const int mb = blockIdx.x / KB, kb = blockIdx.x - mb * KB;
  const int k = kb * 128 + 8 * (threadIdx.x & 15);
  const long long r0 = (long long)mb * 128 + (threadIdx.x >> 4);
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + 16 * i < M && k < K) {
      load8<DT>(x, (r0 + 16 * i) * ldx + k, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  bool special = false;
  unsigned int m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, amax8(v[i], special));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < QZ_THREADS / 32; ++i) m = max(m, wmax[i]);
  const int s = scale_exp(m);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < M && k < K)
      *reinterpret_cast<uint2*>(codes + (r0 + 16 * i) * K + k) = codes8(v[i], s, special);
  if (threadIdx.x == 0) scales[blockIdx.x] = static_cast<uint8_t>(s + 127);
}

template <int DT>
static cudaError_t launch_quantize(const void* x, long long ldx, long long M, int K, int block_rows, uint8_t* codes,
                                   uint8_t* scales, cudaStream_t st) {
  const int KB = (K + 127) / 128;
  if (block_rows == 1) {
    const unsigned int units = static_cast<unsigned int>(M * KB);
    constexpr unsigned int per = QZ_THREADS / 16 * QZ_UNROLL;
    return launch_pdl(quantize_rows_kernel<DT>, dim3((units + per - 1) / per), dim3(QZ_THREADS), 0, st, x, ldx, K, KB,
                      units, codes, scales);
  }
  return launch_pdl(quantize_blocks_kernel<DT>, dim3(static_cast<unsigned int>((M + 127) / 128 * KB)), dim3(QZ_THREADS),
                    0, st, x, ldx, M, K, KB, codes, scales);
}

cudaError_t launch_quantize_fp8(const void* x, int x_dtype, long long ldx, long long M, int K, int block_rows,
                                uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  switch (x_dtype) {
    case SPLICE_F32: return launch_quantize<SPLICE_F32>(x, ldx, M, K, block_rows, codes, scales, st);
    case SPLICE_BF16: return launch_quantize<SPLICE_BF16>(x, ldx, M, K, block_rows, codes, scales, st);
    default: return launch_quantize<SPLICE_F16>(x, ldx, M, K, block_rows, codes, scales, st);
  }
}

// -------------------------------------------------------------------- linear
//
// Scales in tensor memory (kind::mxf8f6f4, one E8M0 byte per row and step):
// row r's byte sits in lane r % 32 of column r / 32, the same in all four
// lane quarters, and the instruction descriptor's scale id picks one of the
// column's four bytes.  A scale here covers 128 elements = four steps, so
// the four bytes hold four k-blocks: one slot of 4 (A) + BN / 32 (B) columns
// serves 512 elements of K.  Four scale warps, one per lane quarter, read
// the bytes from global memory and write them with tcgen05.st, a ring of
// slots ahead of the MMAs; a tcgen05.commit gives each slot back.

namespace {

struct Fp8Params {
  const uint8_t* xs;  // [M, KB] activation scales
  const uint8_t* ws;  // [ceil(N / 128), KB] weight scales
  int KB;
};

template <int BN_>
struct Fp8Shape {
  static constexpr int BM = 128, BN = BN_, BK = 128;
  static constexpr int STAGES = BN >= 128 ? 6 : 8;
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int ACC_COLS = BN;
  static constexpr int SF_A = 4, SF_B = BN / 32, SF_COLS = (SF_A + SF_B + 3) / 4 * 4;  // columns of one scale slot
  static constexpr int SF_SLOTS = 4;
  static constexpr int SF_BASE = 2 * ACC_COLS;
  static constexpr int TMEM_USED = SF_BASE + SF_SLOTS * SF_COLS;
  static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  static constexpr int EPI_WARPS = 8, SF_WARPS = 4;
  static constexpr int THREADS = 32 * (2 + EPI_WARPS + SF_WARPS);
  static constexpr int EPI_BUF_BYTES = EPI_WARPS * 4096;
  static constexpr int BARS = 2 * STAGES + 4 + 2 * SF_SLOTS + 1;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_BUF_BYTES + 8 * BARS + 16;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(TMEM_USED <= 512, "tensor memory");
};

// Instruction descriptor of kind::mxf8f6f4: e4m3 A and B (format 0), K-major,
// E8M0 scales (bit 23); bits 4-5 and 29-30 pick the scale byte of B and A.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N) {
  return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_sf(uint32_t idesc, int byte) {
  return idesc | (static_cast<uint32_t>(byte) << 4) | (static_cast<uint32_t>(byte) << 29);
}
__device__ __forceinline__ void tc_mma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// One 32-bit column of this warp's 32 lanes.
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}

// The four scale bytes of k-blocks 4 g .. 4 g + 3 of one row (1.0 past the end).
__device__ __forceinline__ uint32_t sf_word(const uint8_t* row, int g, int KB, bool valid, bool word_ok) {
  if (!valid) return 0x7F7F7F7Fu;
  if (word_ok) return __ldg(reinterpret_cast<const unsigned int*>(row + 4 * g));
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) w |= (4 * g + j < KB ? static_cast<uint32_t>(__ldg(row + 4 * g + j)) : 0x7Fu) << (8 * j);
  return w;
}

}  // namespace

// One persistent CTA per SM over 128 x BN tiles: warp 0 loads (TMA), warp 1
// issues the MMAs, warps 2-9 run the epilogue of gemm.cuh, warps 10-13 keep
// the scale ring filled.  Waits are bounded; a role that gives up marks the
// CTA in shared memory, and the CTA reports it to p.status at its end.
template <int BN, int EPI, int KIND>
__global__ void __launch_bounds__(Fp8Shape<BN>::THREADS, 1)
    gemm_fp8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmOut, const GemmParams p, const Fp8Params f) {
  using S = Fp8Shape<BN>;
  constexpr int STAGES = S::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int failed;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * S::A_BYTES;
  uint8_t* sEpi = smem + STAGES * S::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + S::EPI_BUF_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* sfull = tempty + 2;
  uint64_t* sempty = sfull + S::SF_SLOTS;
  uint64_t* drain = sempty + S::SF_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    failed = 0;
    for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    for (int a = 0; a < 2; ++a) mbar_init(&tfull[a], 1), mbar_init(&tempty[a], S::EPI_WARPS);
    for (int s = 0; s < S::SF_SLOTS; ++s) mbar_init(&sfull[s], S::SF_WARPS), mbar_init(&sempty[s], 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const int groups = (p.k_blocks + 3) / 4;  // scale slots of a tile

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < p.num_tiles && ok; t += gridDim.x) {
        int mb, nb;
        tile_coords(p, t, mb, nb);
        for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
          const int s = it % STAGES;
          if (!(ok = mbar_wait(&empty[s], ((it / STAGES) & 1) ^ 1, p.limit_ns, &failed, DEV_TIMEOUT_PRODUCER)))
            break;
          mbar_arrive_expect_tx(&full[s], S::STAGE_BYTES);
          tma_load_2d(sA + s * S::A_BYTES, &tmA, &full[s], kb * S::BK, mb * S::BM);
          tma_load_2d(sB + s * S::B_BYTES, &tmB, &full[s], kb * S::BK, nb * BN);
        }
      }
      // every issued load lands before the CTA exits
      for (int s = 0; s < STAGES && s < it; ++s)
        mbar_wait_bounded(&full[s], ((it - 1 - s) / STAGES) & 1, kDrainLimitNs, nullptr, 0);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_mxf8(S::BM, BN);
      int it = 0, tl = 0, sg = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < p.num_tiles && ok; t += gridDim.x, ++tl) {
        const int a = tl & 1;
        if (!(ok = mbar_wait(&tempty[a], ((tl >> 1) & 1) ^ 1, p.limit_ns, &failed, DEV_TIMEOUT_MMA))) break;
        const uint32_t d = tmem + a * S::ACC_COLS;
        for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
          const int s = it % STAGES, slot = sg % S::SF_SLOTS;
          if ((kb & 3) == 0 && !(ok = mbar_wait(&sfull[slot], (sg / S::SF_SLOTS) & 1, p.limit_ns, &failed,
                                                        DEV_TIMEOUT_MMA)))
            break;
          if (!(ok = mbar_wait(&full[s], (it / STAGES) & 1, p.limit_ns, &failed, DEV_TIMEOUT_MMA))) break;
          tc_fence_after();
          const uint64_t ad = sw128_kmajor_desc(smem_u32(sA + s * S::A_BYTES));
          const uint64_t bd = sw128_kmajor_desc(smem_u32(sB + s * S::B_BYTES));
          const uint32_t sf = tmem + S::SF_BASE + slot * S::SF_COLS;
          const uint32_t id = idesc_sf(idesc, kb & 3);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_mxf8(d, ad + 2 * k, bd + 2 * k, id, sf, sf + S::SF_A, (kb > 0 || k > 0) ? 1u : 0u);
          tc_commit(&empty[s]);
          if ((kb & 3) == 3 || kb == p.k_blocks - 1) {
            tc_commit(&sempty[slot]);
            ++sg;
          }
        }
        if (!ok) break;
        tc_commit(&tfull[a]);
      }
      // all issued MMAs complete before tensor memory is released
      tc_commit(drain);
      mbar_wait_bounded(drain, 0, kDrainLimitNs, nullptr, 0);
    }
  } else if (warp < 2 + S::EPI_WARPS) {
    const int q = warp & 3, half = (warp - 2) / 4;
    int tl = 0, gcount = 0;
    for (int t = blockIdx.x; t < p.num_tiles; t += gridDim.x, ++tl) {
      const int a = tl & 1;
      int mb, nb;
      tile_coords(p, t, mb, nb);
      float breg[4];
      load_bias(p, nb * BN, BN, half, lane, breg);
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[a], (tl >> 1) & 1, p.limit_ns, &failed, DEV_TIMEOUT_EPILOGUE)))
        break;
      tc_fence_after();
      const int m0 = mb * S::BM;
      epilogue_warp<EPI, KIND>(p, &tmOut, tmem + (static_cast<uint32_t>(32 * q) << 16) + a * S::ACC_COLS, m0 + 32 * q,
                               min(m0 + 128, p.M), nb * BN, BN, half, lane, sEpi + (warp - 2) * 4096, breg, PIECE_FULL,
                               64, &gcount);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[a]);
    }
    if (lane == 0) bulk_wait0();
  } else {
    const int q = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    // whole words where every row of scales starts on a 4-byte boundary
    const bool word_ok = f.KB % 4 == 0 && ((reinterpret_cast<uintptr_t>(f.xs) | reinterpret_cast<uintptr_t>(f.ws)) & 3) == 0;
    int sg = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < p.num_tiles && ok; t += gridDim.x) {
      int mb, nb;
      tile_coords(p, t, mb, nb);
      for (int g = 0; g < groups; ++g, ++sg) {
        const int slot = sg % S::SF_SLOTS;
        uint32_t w[S::SF_A + S::SF_B];
#pragma unroll
        for (int c = 0; c < S::SF_A; ++c) {
          const int m = mb * S::BM + 32 * c + lane;
          w[c] = sf_word(f.xs + (long long)m * f.KB, g, f.KB, m < p.M, word_ok);
        }
#pragma unroll
        for (int c = 0; c < S::SF_B; ++c) {
          const int n = nb * BN + 32 * c + lane;
          w[S::SF_A + c] = sf_word(f.ws + (long long)(n >> 7) * f.KB, g, f.KB, n < p.N, word_ok);
        }
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sempty[slot], ((sg / S::SF_SLOTS) & 1) ^ 1, p.limit_ns,
                                                             &failed, DEV_TIMEOUT_GATHER))))
          break;
        tc_fence_after();
        const uint32_t dst = tmem + S::SF_BASE + slot * S::SF_COLS + lanes;
#pragma unroll
        for (int c = 0; c < S::SF_A + S::SF_B; ++c) tmem_st1(dst + c, w[c]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[slot]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, S::TMEM_COLS);
  if (threadIdx.x == 0 && failed) atomicCAS(p.status, 0, failed);
}

namespace {

template <int BN, int EPI, int KIND = KIND_BF16>
cudaError_t run_fp8(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o, const GemmParams& p,
                    const Fp8Params& f, int grid, cudaStream_t st) {
  using S = Fp8Shape<BN>;
  auto k = gemm_fp8_tc_kernel<BN, EPI, KIND>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(grid), dim3(S::THREADS), S::SMEM_BYTES, st, a, b, o, p, f);
}

template <int BN>
cudaError_t run_fp8_epi(int epi, bool f16, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                        const GemmParams& p, const Fp8Params& f, int grid, cudaStream_t st) {
  switch (epi) {
    case 0: return f16 ? run_fp8<BN, 0, KIND_F16>(a, b, o, p, f, grid, st) : run_fp8<BN, 0>(a, b, o, p, f, grid, st);
    case EPI_GELU: return run_fp8<BN, EPI_GELU>(a, b, o, p, f, grid, st);
    case EPI_OUT_F32: return run_fp8<BN, EPI_OUT_F32>(a, b, o, p, f, grid, st);
    case EPI_RESID: return run_fp8<BN, EPI_RESID>(a, b, o, p, f, grid, st);
    case EPI_SWIGLU: return run_fp8<BN, EPI_SWIGLU>(a, b, o, p, f, grid, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_linear_fp8(const void* x, const uint8_t* xs, const void* w, const uint8_t* ws, GemmParams p, int epi,
                              bool f16, int num_sms, cudaStream_t st) {
  const bool narrow = (p.M + 127) / 128 * ((p.N + 127) / 128) * 2 <= num_sms;
  const int bn = narrow ? 32 : 128;
  CUtensorMap a, b, o;
  if (!make_tmap_u8(&a, x, p.M, p.K, 128) || !make_tmap_u8(&b, w, p.N, p.K, bn)) return cudaErrorInvalidValue;
  p.out_tma = !(epi & EPI_SWIGLU) && make_tmap_out(&o, p.out, p.M, p.N, p.ldo, (epi & (EPI_OUT_F32 | EPI_RESID)) != 0);
  if (!p.out_tma) o = b;
  p.m_blocks = (p.M + 127) / 128;
  p.n_blocks = (p.N + bn - 1) / bn;
  p.k_blocks = (p.K + 127) / 128;
  p.num_tiles = p.m_blocks * p.n_blocks;
  p.n_fast = p.M > p.N;
  const Fp8Params f = {xs, ws, p.k_blocks};
  const int grid = std::min(p.num_tiles, num_sms);
  return narrow ? run_fp8_epi<32>(epi, f16, a, b, o, p, f, grid, st) : run_fp8_epi<128>(epi, f16, a, b, o, p, f, grid, st);
}

}  // namespace asr
