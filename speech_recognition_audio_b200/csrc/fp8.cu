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
constexpr int QZ_UNROLL = 2;  // blocks of 128 in flight per half-warp (1, 2, 4, 8: 23.3, 19.5, 20.6, 24.7 us at 6240 x 5120 bf16)

// Eight consecutive elements as they are in memory: 16-byte loads (the
// pointer is aligned), two for fp32.
template <int DT>
struct Raw8 {
  static constexpr int W = DT == SPLICE_F32 ? 8 : 4;
  uint32_t w[W];
  __device__ __forceinline__ void load(const void* x, long long i) {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(x) + i * (DT == SPLICE_F32 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
      const uint4 u = __ldg(p + j);
      w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = 0;
  }
  // Largest magnitude as bits of the type, which order like the value
  // (infinities and NaN above all): one word for fp32, the larger of each half
  // of the words for the 16-bit types.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < W; ++j)
      m = DT == SPLICE_F32 ? max(m, w[j] & 0x7FFFFFFFu) : __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    return m;
  }
  // The same over the finite elements only.
  __device__ __forceinline__ uint32_t top_finite() const {
    constexpr uint32_t inf = DT == SPLICE_F32 ? 0x7F800000u : DT == SPLICE_BF16 ? 0x7F80u : 0x7C00u;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if (DT == SPLICE_F32) {
        const uint32_t b = w[j] & 0x7FFFFFFFu;
        m = max(m, b < inf ? b : 0u);
      } else {
        const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
        m = __vmaxu2(m, (lo < inf ? lo : 0u) | (hi < inf ? hi << 16 : 0u));
      }
    }
    return m;
  }
  __device__ __forceinline__ void values(float* v) const {
    if constexpr (DT == SPLICE_F32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    } else {
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
};
template <int DT>
__device__ __forceinline__ uint32_t top_max(uint32_t a, uint32_t b) {
  return DT == SPLICE_F32 ? max(a, b) : __vmaxu2(a, b);
}
// fp32 bits of the magnitude that top() describes; whether it is not finite.
template <int DT>
__device__ __forceinline__ uint32_t top_bits(uint32_t m) {
  if constexpr (DT == SPLICE_F32) return m;
  const uint32_t h = max(m & 0xFFFFu, m >> 16);
  if constexpr (DT == SPLICE_BF16) return h << 16;
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}
__device__ __forceinline__ bool bits_special(uint32_t b) { return b >= 0x7F800000u; }

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
template <int DT>
__device__ __forceinline__ uint2 codes8(const Raw8<DT>& r, int s, bool special) {
  float v[8];
  r.values(v);
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
// segment per block).  Bound by HBM: 27.6 us for 48000 x 768 fp32 (184 MB, the
// copy rate), 19.0 for 6240 x 5120 bf16 (96 MB).
template <int DT>
__global__ void __launch_bounds__(QZ_THREADS) quantize_rows_kernel(const void* __restrict__ x, long long ldx, int K,
                                                                   int KB, unsigned int units,
                                                                   uint8_t* __restrict__ codes,
                                                                   uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int l16 = threadIdx.x & 15;
  const unsigned int first = blockIdx.x * (QZ_THREADS / 16 * QZ_UNROLL) + (threadIdx.x >> 4);
  Raw8<DT> v[QZ_UNROLL];
  unsigned int row[QZ_UNROLL];
  int kb[QZ_UNROLL];
#pragma unroll
  for (int i = 0; i < QZ_UNROLL; ++i) {
    const unsigned int u = first + i * (QZ_THREADS / 16);
    row[i] = u / static_cast<unsigned int>(KB);
    kb[i] = static_cast<int>(u - row[i] * KB);
    const int k = kb[i] * 128 + 8 * l16;
    if (u < units && k < K)
      v[i].load(x, row[i] * ldx + k);
    else
      v[i].clear();
  }
#pragma unroll
  for (int i = 0; i < QZ_UNROLL; ++i) {
    const unsigned int u = first + i * (QZ_THREADS / 16);
    auto over_block = [](uint32_t m) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m = top_max<DT>(m, __shfl_xor_sync(0xffffffffu, m, o));
      return top_bits<DT>(m);
    };
    uint32_t m = over_block(v[i].top());
    const bool special = bits_special(m);
    if (__any_sync(0xffffffffu, special)) {  // rare: the scale goes by the finite values
      const uint32_t f = over_block(v[i].top_finite());
      if (special) m = f;
    }
    const int s = scale_exp(m);
    const int k = kb[i] * 128 + 8 * l16;
    if (u < units) {
      if (k < K) *reinterpret_cast<uint2*>(codes + (long long)row[i] * K + k) = codes8<DT>(v[i], s, special);
      if (l16 == 0) scales[u] = static_cast<uint8_t>(s + 127);
    }
  }
}

// One scale per 128 x 128 block (weights): one thread block each, the 128
// rows in eight passes of sixteen, held in registers between the maximum and
// the conversion.  Bound by HBM: 27.6 us for 16384 x 2048 fp32 (168 MB, 93 % of
// the copy rate), 16.9 for bf16 (101 MB).
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
  Raw8<DT> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + 16 * i < M && k < K)
      v[i].load(x, (r0 + 16 * i) * ldx + k);
    else
      v[i].clear();
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = top_max<DT>(m, v[i].top());
  auto over_block = [&](uint32_t bits) {
    bits = __reduce_max_sync(0xffffffffu, bits);
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = bits;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < QZ_THREADS / 32; ++i) bits = max(bits, wmax[i]);
    return bits;
  };
  uint32_t top = over_block(top_bits<DT>(m));
  const bool special = bits_special(top);
  if (special) {  // rare, the whole block together: the scale goes by the finite values
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = top_max<DT>(m, v[i].top_finite());
    __syncthreads();  // wmax has been read
    top = over_block(top_bits<DT>(m));
  }
  const int s = scale_exp(top);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < M && k < K)
      *reinterpret_cast<uint2*>(codes + (r0 + 16 * i) * K + k) = codes8<DT>(v[i], s, special);
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

template <int EPI>
constexpr bool epi_wide() {  // 16-bit outputs stored as they are: 64 columns = 128-byte rows
  return (EPI & ~EPI_GELU) == 0;
}

template <int BN_, bool WIDE>
struct Fp8Shape {
  static constexpr int BM = 128, BN = BN_, BK = 128;
  static constexpr int STAGES = BN == 192 ? 4 : BN == 128 ? 5 : 8;
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int ACC_COLS = BN;
  static constexpr int SF_A = 4, SF_B = BN / 32, SF_COLS = (SF_A + SF_B + 3) / 4 * 4;  // columns of one scale slot
  static constexpr int SF_SLOTS = 4;
  static constexpr int SF_BASE = 2 * ACC_COLS;
  static constexpr int TMEM_USED = SF_BASE + SF_SLOTS * SF_COLS;
  static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  // epilogue warps: four per 64 columns (wide), or two column parts of 32-column groups
  static constexpr int PARTS = !WIDE ? 2 : (BN + 63) / 64, EPI_WARPS = 4 * PARTS, SF_WARPS = 4;
  static constexpr int THREADS = 32 * (2 + EPI_WARPS + SF_WARPS);
  static constexpr int EPI_BUF_BYTES = EPI_WARPS * 4096;
  static constexpr int BARS = 2 * STAGES + 4 + 2 * SF_SLOTS + 1;
  static constexpr int BIAS_BYTES = WIDE ? EPI_WARPS * 256 : 0;
  static constexpr int SF_DEPTH = 8, SF_ROWS = 128 + 8, SF_BYTES = SF_DEPTH * SF_ROWS * 8;  // scale bytes on their way
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_BUF_BYTES + BIAS_BYTES + SF_BYTES + 8 * BARS + 16;
  static_assert(SMEM_BYTES <= 227 * 1024 - 16, "shared memory");
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
// The four K = 32 steps of a 128-element k-block.  Written for a whole warp in
// step, one elected lane issuing: 6240 x 1280 x 5120 took 40 us this way and
// 86 with a branch that only one lane took.
__device__ __forceinline__ void tc_mma4_mxf8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t accumulate) {
  asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %7, %8, %3, [%5], [%6], 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %9, %10, %3, [%5], [%6], 1;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %11, %12, %3, [%5], [%6], 1;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "l"(ad + 2), "l"(bd + 2), "l"(ad + 4),
        "l"(bd + 4), "l"(ad + 6), "l"(bd + 6)
        : "memory");
}
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Barrier of the four scale warps.
__device__ __forceinline__ void sf_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// One 32-bit column of this warp's 32 lanes.
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}

// Starts the copy of the scale bytes of k-blocks 4 g .. 4 g + 3 of row r of
// scales [rows, KB] to dst: the aligned words around them (a row of whole
// words fills only the first), from which sf_bytes picks them.  Where a word
// would reach past the array, or the array is not aligned, bytes are read one
// by one.  What follows the row's last byte is never used.
__device__ __forceinline__ void sf_copy(uint2* dst, const uint8_t* sc, long long r, long long rows, int g, int KB, bool aligned) {
  const long long off = r * KB + 4 * g;
  const int sh = static_cast<int>(off & 3);
  if (aligned && off - sh + (sh ? 8 : 4) <= rows * KB) {
    cp_async_4(&dst->x, sc + (off - sh));
    if (sh) cp_async_4(&dst->y, sc + (off - sh) + 4);
  } else {
    uint64_t v = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * g + j < KB) v |= static_cast<uint64_t>(__ldg(sc + off + j)) << (8 * (sh + j));
    *dst = make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
  }
}
__device__ __forceinline__ uint32_t sf_bytes(uint2 v, long long r, int KB) {
  return __funnelshift_r(v.x, v.y, 8 * static_cast<int>(r * KB & 3));
}

// Epilogue of one warp for 16-bit outputs: its 32 rows and COLS (64, or
// a 32-wide tile's 32) columns are read
// into registers at once (the accumulator goes back to the MMAs before any of
// the arithmetic), get bias and GELU, and leave as one TMA store of 128-byte
// rows.  (48000 x 18432 x 768 on 128 x 128 tiles: 1141 us through the engine's
// epilogue, whose boxes are 32 columns and which holds the accumulator
// throughout; 842 us this way, with the scales loaded as below.)
template <int COLS, int EPI, int KIND, typename Release>
__device__ __forceinline__ void epilogue_wide(const GemmParams& p, const CUtensorMap* tm_out, uint32_t taddr, int row0,
                                              int n, int lane, uint8_t* buf, const float* bias,
                                              Release release) {
  float v[COLS];
#pragma unroll
  for (int c = 0; c < COLS; c += 32) tmem_ld32(taddr + c, v + c);
  tmem_ld_wait();
  tc_fence_before();
  __syncwarp();
  release();
  if (row0 >= p.M || n >= p.N) return;  // the whole warp
  if (p.bias) {
#pragma unroll
    for (int k = 0; k < COLS / 4; ++k) {
      const float4 b = reinterpret_cast<const float4*>(bias)[k];  // the same address in every lane
      v[4 * k] += b.x, v[4 * k + 1] += b.y, v[4 * k + 2] += b.z, v[4 * k + 3] += b.w;
    }
  }
  if constexpr ((EPI & EPI_GELU) != 0) {
#pragma unroll
    for (int k = 0; k < COLS; k += 2) {
      const float2 g = gelu_erf2(make_float2(v[k], v[k + 1]));
      v[k] = g.x, v[k + 1] = g.y;
    }
  }
  // the store that last used this buffer has read it
  if (lane == 0) bulk_wait_read0();
  __syncwarp();
  // the 128-byte (or, for 32 columns, 64-byte) swizzle of the store
  uint4* row = reinterpret_cast<uint4*>(buf + lane * (2 * COLS));
  const int x = COLS == 64 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
  for (int k = 0; k < COLS / 8; ++k) row[k ^ x] = pack8_16<KIND>(v + 8 * k);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(tm_out, buf, n, row0);
    bulk_commit();
  }
}

}  // namespace

// One persistent CTA per SM over 128 x BN tiles: warp 0 loads (TMA), warp 1
// issues the MMAs, then come the epilogue warps (four per 64 columns for plain
// 16-bit outputs, else the eight of gemm.cuh's epilogue) and four that keep
// the scale ring filled.  Waits are bounded; a role that gives up marks the
// CTA in shared memory, and the CTA reports it to p.status at its end.
//
// What bounds it: a k-block of a 128 x 192 tile is 384 clocks of MMAs, 40 KB
// into shared memory and 40 KB out of it again.  In a steady loop under the
// power cap 6240 x 2048 x 8192 takes 99 us at 1.49 GHz: 2115 TFLOP/s (65 % of
// twice the measured bf16 rate), 576 clocks a k-block over its four waves of
// 64.  48000 x 18432 x 768 (1.77 GB of output) takes 815-840 us at 1.4 GHz,
// 1640 TFLOP/s, and 750 in the first passes from idle: about 4800 clocks a
// tile of six k-blocks, of which some 1300 are not the main loop's; where they
// go has not been measured.  6240 x 1280 x 5120 with the residual takes 43 us
// from L2 and 47-52 with inputs that change, at 1.97 GHz: three waves of tiles
// where 2.3 would do.
template <int BN, int EPI, int KIND>
__global__ void __launch_bounds__(Fp8Shape<BN, epi_wide<EPI>()>::THREADS, 1)
    gemm_fp8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmOut, const GemmParams p, const Fp8Params f) {
  using S = Fp8Shape<BN, epi_wide<EPI>()>;
  constexpr int STAGES = S::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int failed;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * S::A_BYTES;
  uint8_t* sEpi = smem + STAGES * S::STAGE_BYTES;
  float* sBias = reinterpret_cast<float*>(sEpi + S::EPI_BUF_BYTES);
  uint2* sSf = reinterpret_cast<uint2*>(sEpi + S::EPI_BUF_BYTES + S::BIAS_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + S::EPI_BUF_BYTES + S::BIAS_BYTES + S::SF_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* sfull = tempty + 2;
  uint64_t* sempty = sfull + S::SF_SLOTS;
  uint64_t* drain = sempty + S::SF_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

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
        mbar_wait(&full[s], ((it - 1 - s) / STAGES) & 1, kDrainLimitNs, nullptr, 0);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_mxf8(S::BM, BN);
    const uint64_t ad0 = sw128_kmajor_desc(smem_u32(sA)), bd0 = sw128_kmajor_desc(smem_u32(sB));
    auto wait = [&](uint64_t* b, int n) {
      return __all_sync(0xffffffffu, mbar_wait(b, n & 1, p.limit_ns, &failed, DEV_TIMEOUT_MMA)) != 0;
    };
    int it = 0, tl = 0, sg = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < p.num_tiles && ok; t += gridDim.x, ++tl) {
      const int a = tl & 1;
      if (!(ok = wait(&tempty[a], (tl >> 1) ^ 1))) break;
      const uint32_t d = tmem + a * S::ACC_COLS;
      for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
        const int s = it % STAGES, slot = sg % S::SF_SLOTS;
        if ((kb & 3) == 0 && !(ok = wait(&sfull[slot], sg / S::SF_SLOTS))) break;
        if (!(ok = wait(&full[s], it / STAGES))) break;
        tc_fence_after();
        const uint32_t sf = tmem + S::SF_BASE + slot * S::SF_COLS;
        tc_mma4_mxf8(d, ad0 + s * (S::A_BYTES >> 4), bd0 + s * (S::B_BYTES >> 4), idesc_sf(idesc, kb & 3), sf,
                            sf + S::SF_A, kb > 0 ? 1u : 0u);
        tc_commit_warp(&empty[s]);
        if ((kb & 3) == 3 || kb == p.k_blocks - 1) {
          tc_commit_warp(&sempty[slot]);
          ++sg;
        }
      }
      if (!ok) break;
      tc_commit_warp(&tfull[a]);
    }
    // all issued MMAs complete before tensor memory is released
    tc_commit_warp(drain);
    mbar_wait(drain, 0, kDrainLimitNs, nullptr, 0);
  } else if (warp < 2 + S::EPI_WARPS) {
    const int q = warp & 3, part = (warp - 2) / 4;
    int tl = 0, gcount = 0;
    for (int t = blockIdx.x; t < p.num_tiles; t += gridDim.x, ++tl) {
      const int a = tl & 1;
      int mb, nb;
      tile_coords(p, t, mb, nb);
      const int m0 = mb * S::BM;
      const uint32_t acc = tmem + (static_cast<uint32_t>(32 * q) << 16) + a * S::ACC_COLS;
      uint8_t* buf = sEpi + (warp - 2) * 4096;
      auto wait = [&] {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(&tfull[a], (tl >> 1) & 1, p.limit_ns, &failed, DEV_TIMEOUT_EPILOGUE));
        tc_fence_after();
        return ok;
      };
      auto release = [&] {
        if (lane == 0) mbar_arrive(&tempty[a]);
      };
      if constexpr (epi_wide<EPI>()) {
        // the columns' biases, fetched while the accumulator is not ready
        constexpr int COLS = BN < 64 ? BN : 64;
        float* bias = sBias + (warp - 2) * 64;
        const int n = nb * BN + 64 * part;
        __syncwarp();  // the last tile's biases have been read
        if (p.bias) {
          for (int c = lane; c < COLS; c += 32) bias[c] = n + c < p.N ? __ldg(p.bias + n + c) : 0.f;
        }
        __syncwarp();
        if (!wait()) break;
        epilogue_wide<COLS, EPI, KIND>(p, &tmOut, acc + 64 * part, m0 + 32 * q, n, lane,
                                       buf, bias, release);
      } else {
        if (EPI & EPI_RESID) epilogue_prefetch_l2(p, t, part, q, lane, BN, S::BM, 0);
        float breg[4];
        load_bias(p, nb * BN, BN, part, lane, breg);
        if (!wait()) break;
        epilogue_warp<EPI, KIND>(p, &tmOut, acc, m0 + 32 * q, min(m0 + 128, p.M), nb * BN, BN, part, lane, buf, breg,
                                 PIECE_FULL, 64, &gcount);
        tc_fence_before();
        __syncwarp();
        release();
      }
    }
    if (lane == 0) bulk_wait0();
  } else {
    // Scales.  The four warps share out the bytes of a slot (32 rows of A each,
    // the first also B's) as asynchronous copies, SF_DEPTH slots ahead, and
    // each writes all of them to its own lane quarter.  The depth is what
    // matters: beside the output's writes a load takes over 2000 clocks, and
    // loading one or two slots ahead left the MMAs waiting 2600 clocks a tile.
    const int q = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const bool xs_al = (reinterpret_cast<uintptr_t>(f.xs) & 3) == 0, ws_al = (reinterpret_cast<uintptr_t>(f.ws) & 3) == 0;
    const int items = p.num_tiles > (int)blockIdx.x ? ((p.num_tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1) * groups : 0;
    struct Item {  // the k-th (tile, slot) of this block
      int t, g, mb, nb;
    };
    auto advance = [&](Item& i) {
      if (++i.g == groups) {
        i.g = 0;
        i.t += gridDim.x;
        tile_coords(p, i.t, i.mb, i.nb);
      }
    };
    Item ahead = {static_cast<int>(blockIdx.x), 0, 0, 0};
    tile_coords(p, ahead.t, ahead.mb, ahead.nb);
    Item cur = ahead;
    int n_ahead = 0;
    auto copy = [&] {  // one group per call, empty past the end
      if (n_ahead < items) {
        uint2* dst = sSf + n_ahead % S::SF_DEPTH * S::SF_ROWS;
        const int m = ahead.mb * S::BM + 32 * q + lane, n = ahead.nb * BN + 32 * lane;
        if (m < p.M) sf_copy(dst + 32 * q + lane, f.xs, m, p.M, ahead.g, f.KB, xs_al);
        // a column's 32 rows of B share one 128-row block
        if (q == 0 && lane < S::SF_B && n < p.N) sf_copy(dst + 128 + lane, f.ws, n >> 7, (p.N + 127) / 128, ahead.g, f.KB, ws_al);
        advance(ahead);
        ++n_ahead;
      }
      cp_async_commit();
    };
    for (int i = 0; i < S::SF_DEPTH - 1; ++i) copy();
    // After a failed wait the loop runs on without waiting: the four warps
    // meet the same barriers.
    bool ok = true;
    for (int i = 0; i < items; ++i) {
      cp_async_wait<S::SF_DEPTH - 2>();
      sf_sync();  // slot i has arrived, slot i - 1 has been read by all
      copy();
      const uint2* src = sSf + i % S::SF_DEPTH * S::SF_ROWS;
      uint32_t w[S::SF_A + S::SF_B];
#pragma unroll
      for (int c = 0; c < S::SF_A; ++c) {
        const int m = cur.mb * S::BM + 32 * c + lane;
        // rows past the end: any finite scale
        w[c] = m < p.M ? sf_bytes(src[32 * c + lane], m, f.KB) : 0x7F7F7F7Fu;
      }
#pragma unroll
      for (int c = 0; c < S::SF_B; ++c) {
        const int n = cur.nb * BN + 32 * c;
        w[S::SF_A + c] = n < p.N ? sf_bytes(src[128 + c], n >> 7, f.KB) : 0x7F7F7F7Fu;
      }
      advance(cur);
      const int slot = i % S::SF_SLOTS;
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&sempty[slot], ((i / S::SF_SLOTS) & 1) ^ 1, p.limit_ns, &failed,
                                                   DEV_TIMEOUT_GATHER));
      tc_fence_after();
      const uint32_t dst = tmem + S::SF_BASE + slot * S::SF_COLS + lanes;
#pragma unroll
      for (int c = 0; c < S::SF_A + S::SF_B; ++c) tmem_st1(dst + c, w[c]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&sfull[slot]);
    }
    cp_async_wait_all();
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
  using S = Fp8Shape<BN, epi_wide<EPI>()>;
  auto k = gemm_fp8_tc_kernel<BN, EPI, KIND>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_once(k, S::SMEM_BYTES, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(grid), dim3(S::THREADS), S::SMEM_BYTES, st, a, b, o, p, f);
}

template <int BN>
cudaError_t run_fp8_epi(int epi, bool f16, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                        const GemmParams& p, const Fp8Params& f, int grid, cudaStream_t st) {
  switch (epi) {
    case 0:
      return f16 ? run_fp8<BN, 0, KIND_F16>(a, b, o, p, f, grid, st) : run_fp8<BN, 0>(a, b, o, p, f, grid, st);
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
  // The tile width with the least waves x time of a tile, 20 : 25 : 29 a
  // k-block of a 128 x 32, 128 or 192 tile alone on its SM (64 x 1280 x 5120:
  // 10.6, 11.3 and 13.1 us); wider ones move fewer bytes per product and win
  // once every SM has work.  Measured, us, bf16 outputs, inputs that change:
  // 6240 x 1280 x 5120 114, 42.7, 41.8; 5 x 768 x 768 3.9, 4.3, 4.8; 780 x 1280
  // x 1280 7.5, 5.8, 6.7.  CTA pairs (256 x 192) were slower throughout: 53.7
  // at 6240 x 1280 x 5120, where 192 took 38.0 on the same inputs.
  const int mb = (p.M + 127) / 128;
  int bn = 0;
  long long least = 0;
  for (const auto& c : {std::pair<int, int>{32, 20}, {128, 25}, {192, 29}}) {
    const long long waves = ((long long)mb * ((p.N + c.first - 1) / c.first) + num_sms - 1) / num_sms;
    if (!bn || waves * c.second < least) bn = c.first, least = waves * c.second;
  }
  CUtensorMap a, b, o;
  if (!make_tmap_u8(&a, x, p.M, p.K, 128) || !make_tmap_u8(&b, w, p.N, p.K, bn)) return cudaErrorInvalidValue;
  if ((epi & ~EPI_GELU) == 0) {
    if (!(bn == 32 ? make_tmap_out(&o, p.out, p.M, p.N, p.ldo, false) : make_tmap_bf16(&o, p.out, p.M, p.N, p.ldo, 32)))
      return cudaErrorInvalidValue;
  } else {
    p.out_tma = !(epi & EPI_SWIGLU) && make_tmap_out(&o, p.out, p.M, p.N, p.ldo, true);
    if (!p.out_tma) o = b;
  }
  p.m_blocks = mb;
  p.n_blocks = (p.N + bn - 1) / bn;
  p.k_blocks = (p.K + 127) / 128;
  p.num_tiles = p.m_blocks * p.n_blocks;
  p.n_fast = p.M > p.N;
  const Fp8Params f = {xs, ws, p.k_blocks};
  const int grid = std::min(p.num_tiles, num_sms);
  switch (bn) {
    case 32: return run_fp8_epi<32>(epi, f16, a, b, o, p, f, grid, st);
    case 128: return run_fp8_epi<128>(epi, f16, a, b, o, p, f, grid, st);
    default: return run_fp8_epi<192>(epi, f16, a, b, o, p, f, grid, st);
  }
}

}  // namespace asr
