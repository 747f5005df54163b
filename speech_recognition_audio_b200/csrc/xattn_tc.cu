// Cross attention of many rows on the tcgen05 tensor cores.
//
// One block takes a tile of 128 rows of one (segment, head) over the segment's
// states in tiles of 128; two blocks share an SM:
//   warp 8    TMA: the query tile once, then K_j and V_j into rings;
//   warp 9    MMA: S = Q K_j^T (128 x 128 x 64), then O += P V_j
//             (128 x 64 x 128) with P read from tensor memory;
//   warps 0-7 softmax: warps w and w + 4 share the 32 rows of lane quarter
//             w % 4 and take 64 of the tile's states and 32 of O's columns
//             each; a thread reads its 64 scores into registers at once, so
//             the next tile's product runs under the exponentials.
// Tensor memory: S 128, P 64, O 64 columns, none shared.
//
// Floors: 16 exponentials per clock and SM against 4096 products, so a tile of
// 128 x 128 costs 1024 clocks of them and 512 of the tensor pipe.  2240 rows x
// 1500 states x 12 heads x 32 segments (330 GFLOP, 1.29e9 exponentials = 277 us
// at 1965 MHz): 600-613 us, 540-550 TFLOP/s.  What bounds it is the chain of a step
// (wait, read, maximum, exponentials, write, product), of which four softmax
// warps per scheduler hide about half: the exponential unit is 52 % busy, the
// tensor pipe 25 %, issue 48 %.  Measured on the way there: single-lane issue with
// waits behind a call 868; one thread a row and two tiles a block 617, with
// the tiles' exponentials taking turns 762; exponentials ahead of the maximum,
// repeated where it moved, 615; two independent streams of 64-state tiles a
// block, P over S, 626; persistent blocks running ahead into the next tile of
// rows, with two K tiles in flight, 681.
//
// The running maximum used for the exponentials moves only when a row's
// maximum exceeds it by more than 2^8 (then O and the sum are rescaled), so
// probabilities stay below 2^8 and most tiles need no rescale.  Sums are kept
// in fp32 from the unrounded probabilities; a probability is rounded once, to
// the values' type, as the tensor core's operand.
//
// With few blocks the states are split over the blocks of a cluster: each
// leaves its O, maximum and sum in shared memory, and the rows are joined in
// rank order through distributed shared memory.
#include "xattn.cuh"

namespace asr {

namespace {

constexpr float kRescaleLog2 = 8.0f;
// whole warpgroups, so that registers can move from the load and issue warps
// to the softmax; the sum stays within the launch's 384 x 80 (two blocks per SM)
constexpr int XT_THREADS = 384, XT_TMA_WARP = 8, XT_MMA_WARP = 9;
constexpr int XT_REGS_ISSUE = 32, XT_REGS_SOFTMAX = 104;
static_assert(128 * XT_REGS_ISSUE + 256 * XT_REGS_SOFTMAX <= XT_THREADS * 80, "registers");
// K and V tiles in flight (two blocks per SM leave 113 KB each)
constexpr int XT_KS = 3, XT_VS = 2, XT_TILE = 16384;
constexpr int XT_SQ = 0, XT_SK = XT_TILE, XT_SV = XT_SK + XT_KS * XT_TILE, XT_RED = XT_SV + XT_VS * XT_TILE;
constexpr int XT_BARS = XT_RED + 2 * 2 * 128 * 4;  // after the halves' maxima [2][2][128]
enum { XB_Q = 0, XB_KF, XB_KE = XB_KF + XT_KS, XB_VF = XB_KE + XT_KS, XB_VE = XB_VF + XT_VS, XB_SF = XB_VE + XT_VS,
       XB_SE, XB_PF, XB_OD, XB_DRAIN, XB_COUNT };
constexpr int XT_SMEM = 1024 + XT_BARS + 8 * XB_COUNT + 16;
constexpr int XT_S = 0, XT_P = 128, XT_O = 192, XT_TMEM_COLS = 256;
// the parts of a split row reuse the tiles: 64 floats of O (row padded to 68), then maximum and sum
constexpr int XT_PART_LD = 68;
static_assert(128 * (XT_PART_LD + 2) * 4 <= XT_RED, "parts fit in the tiles");
static_assert(2 * (XT_SMEM + 1024) <= 228 * 1024, "two blocks per SM");

// The tensor-core issue below is written for a whole warp in step: every lane
// computes the same addresses and one elected lane issues.  The rescoring case
// took 651 us this way and 719 with a branch that only one lane took.
// S = Q K^T: the four K = 16 steps of 64 elements.
__device__ __forceinline__ void tc_scores_warp(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %5, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %6, %7, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %8, %9, %3, 1;\n\t}" ::"r"(d_tmem),
      "l"(ad), "l"(bd), "r"(idesc), "l"(ad + 2), "l"(bd + 2), "l"(ad + 4), "l"(bd + 4), "l"(ad + 6), "l"(bd + 6)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], four K = 16 steps: A's rows are lanes, two
// 16-bit elements of K per column (8 columns a step); B = 16 rows of V a step.
__device__ __forceinline__ void tc_values_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t bd, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %6, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %8, %3, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%9], %10, %3, 1;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bd), "r"(idesc), "r"(accumulate), "r"(a_tmem + 8), "l"(bd + 128), "r"(a_tmem + 16), "l"(bd + 256),
      "r"(a_tmem + 24), "l"(bd + 384)
      : "memory");
}
// Barriers of the two softmax warps of a lane quarter (ids 1-4) and of the
// whole block, reached from different branches (id 5).
__device__ __forceinline__ void pair_sync(int q) { asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory"); }
__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 5, %0;" ::"n"(XT_THREADS) : "memory"); }

}  // namespace

template <int KIND>
__global__ void __launch_bounds__(XT_THREADS, 2)
    xattn_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const XattnArgs a, int q_blocks) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int failed;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(sm + XT_RED);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + XT_BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + XB_COUNT);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    failed = 0;
    for (int i = 0; i < XB_COUNT; ++i) mbar_init(&bar[i], i == XB_SE || i == XB_PF ? 8 : 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == XT_MMA_WARP) {
    tmem_alloc(tmem_slot, XT_TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int S = a.splits, rank = blockIdx.x % S, unit = blockIdx.x / S;
  const int seg = unit / q_blocks, row0 = (unit - seg * q_blocks) * 128, h = blockIdx.y, kvh = h / a.G;
  const Segment s = load_segment(a, seg, tid == 0);
  const bool live = s.ok && row0 < s.lq;  // the same for every block of the cluster
  // this block's tiles of states
  const int tiles = (s.lk + 127) / 128;
  const int t0 = (int)((long long)rank * tiles / S), nk = (int)((long long)(rank + 1) * tiles / S) - t0;

  if (warp >= XT_TMA_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(XT_REGS_ISSUE));
    if (!live) {
    } else if (nk > 0 && warp == XT_TMA_WARP) {
      if (lane == 0) {
        const int k0 = s.k0 + t0 * 128;
        mbar_arrive_expect_tx(&bar[XB_Q], XT_TILE);
        tma_load_2d(sm + XT_SQ, &tm_q, &bar[XB_Q], h * 64, s.q0 + row0);
        int nkl = 0, nvl = 0;
        for (int j = 0; j < nk; ++j) {
          const int ks = j % XT_KS, vs = j % XT_VS;
          if (!mbar_wait(&bar[XB_KE + ks], ((j / XT_KS) & 1) ^ 1, a.limit_ns, &failed, DEV_TIMEOUT_PRODUCER)) break;
          mbar_arrive_expect_tx(&bar[XB_KF + ks], XT_TILE);
          tma_load_2d(sm + XT_SK + ks * XT_TILE, &tm_k, &bar[XB_KF + ks], kvh * 64, k0 + j * 128);
          ++nkl;
          if (!mbar_wait(&bar[XB_VE + vs], ((j / XT_VS) & 1) ^ 1, a.limit_ns, &failed, DEV_TIMEOUT_PRODUCER)) break;
          mbar_arrive_expect_tx(&bar[XB_VF + vs], XT_TILE);
          tma_load_2d(sm + XT_SV + vs * XT_TILE, &tm_v, &bar[XB_VF + vs], kvh * 64, k0 + j * 128);
          ++nvl;
        }
        // every issued load lands before the shared memory is reused or left
        mbar_wait(&bar[XB_Q], 0, kDrainLimitNs, nullptr, 0);
        for (int j = max(0, nkl - XT_KS); j < nkl; ++j)
          mbar_wait(&bar[XB_KF + j % XT_KS], (j / XT_KS) & 1, kDrainLimitNs, nullptr, 0);
        for (int j = max(0, nvl - XT_VS); j < nvl; ++j)
          mbar_wait(&bar[XB_VF + j % XT_VS], (j / XT_VS) & 1, kDrainLimitNs, nullptr, 0);
      }
    } else if (nk > 0 && warp == XT_MMA_WARP) {
      const uint32_t idesc_s = idesc_kind_f32(KIND, 128, 128);
      const uint32_t idesc_o = idesc_kind_f32(KIND, 128, 64) | (1u << 16);  // B = V, MN-major
      const uint64_t qd = sw128_kmajor_desc(smem_u32(sm + XT_SQ)), kd = sw128_kmajor_desc(smem_u32(sm + XT_SK));
      const uint64_t vd = sw128_mnmajor_desc(smem_u32(sm + XT_SV));
      auto wait = [&](int b, int n) {
        return __all_sync(0xffffffffu, mbar_wait(&bar[b], n & 1, a.limit_ns, &failed, DEV_TIMEOUT_MMA)) != 0;
      };
      auto issue_s = [&](int j) {
        tc_fence_after();
        tc_scores_warp(tmem + XT_S, qd, kd + (j % XT_KS) * (XT_TILE >> 4), idesc_s);
        tc_commit_warp(&bar[XB_SF]);
        tc_commit_warp(&bar[XB_KE + j % XT_KS]);
      };
      bool ok = wait(XB_Q, 0) && wait(XB_KF, 0);
      if (ok) issue_s(0);
      for (int j = 0; j < nk && ok; ++j) {
        if (j + 1 < nk) {
          // the next scores, once the softmax holds these in registers
          if (!(ok = wait(XB_KF + (j + 1) % XT_KS, (j + 1) / XT_KS) && wait(XB_SE, j))) break;
          issue_s(j + 1);
        }
        if (!(ok = wait(XB_PF, j) && wait(XB_VF + j % XT_VS, j / XT_VS))) break;
        tc_fence_after();
        const uint64_t vj = vd + (j % XT_VS) * (XT_TILE >> 4);
        tc_values_warp(tmem + XT_O, tmem + XT_P, vj, idesc_o, j > 0 ? 1u : 0u);
        tc_values_warp(tmem + XT_O, tmem + XT_P + 32, vj + 512, idesc_o, 1u);
        tc_commit_warp(&bar[XB_OD]);
        tc_commit_warp(&bar[XB_VE + j % XT_VS]);
      }
      // all issued MMAs complete before tensor or shared memory is released
      tc_commit_warp(&bar[XB_DRAIN]);
      mbar_wait(&bar[XB_DRAIN], 0, kDrainLimitNs, nullptr, 0);
    }
    if (S > 1 && live) {  // the softmax warps' side of these is below
      __syncwarp();
      block_sync();
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(XT_REGS_SOFTMAX));
    if (live) {
    const int q = warp & 3, hh = warp >> 2, row = 32 * q + lane;  // lane quarter, half of the states and of O
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float m_used = -INFINITY, lsum = 0.f;  // the row's maximum, this half's sum
    // After a failed wait the loop runs on without waiting, so that the two
    // warps of a pair always meet the same barriers.
    bool ok = true;
    auto wait = [&](int b, int n) {
      ok = ok && mbar_wait(&bar[b], n & 1, a.limit_ns, &failed, DEV_TIMEOUT_EPILOGUE);
      tc_fence_after();
    };
    for (int j = 0; j < nk; ++j) {
      wait(XB_SF, j);
      float sv[64];
      tmem_ld32(trow + XT_S + 64 * hh, sv);
      tmem_ld32(trow + XT_S + 64 * hh + 32, sv + 32);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[XB_SE]);
      const int kv = s.lk - (t0 + j) * 128;  // states left
      if (kv < 128) {
        // scores past the end never count, and values past it, which may be
        // anything (another segment's), become zeros: 0 * NaN would stay NaN
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (64 * hh + c >= kv) sv[c] = -INFINITY;
        if (hh == 0) {
          wait(XB_VF + j % XT_VS, j / XT_VS);
          uint4* rows = reinterpret_cast<uint4*>(sm + XT_SV + (j % XT_VS) * XT_TILE);
          for (int i = kv * 8 + tid; i < 1024; i += 128) rows[i] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
      }
      // The row's maximum over both halves.  Buffers alternate: a warp writes
      // one again only after its partner has passed the next barrier, having
      // read it.
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; c += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], fmaxf(sv[c + 2 * i], sv[c + 2 * i + 1]));
      }
      float* rbuf = red + (j & 1) * 256;
      rbuf[hh * 128 + row] = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      pair_sync(q);
      const float mt = fmaxf(rbuf[row], rbuf[128 + row]) * kScaleLog2;
      const bool grow = mt > m_used + kRescaleLog2;
      if (__any_sync(0xffffffffu, grow)) {
        const float corr = grow ? ex2_approx(m_used - mt) : 1.0f;  // 0 where there was no maximum yet
        if (grow) m_used = mt;
        lsum *= corr;
        if (j > 0) {
          wait(XB_OD, j - 1);  // O is still once the previous product is complete
#pragma unroll
          for (int c = 0; c < 32; c += 16) {
            float ov[16];
            tmem_ld16(trow + XT_O + 32 * hh + c, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) ov[i] *= corr;
            tmem_st16(trow + XT_O + 32 * hh + c, ov);
          }
        }
      }
      const float sh = shift_of(m_used);
      const float2 scale2 = make_float2(kScaleLog2, kScaleLog2), shift2 = make_float2(-sh, -sh);
      float2 s2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
      float pk[32];
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 x = fma2(make_float2(sv[c], sv[c + 1]), scale2, shift2);
        const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        s2[(c >> 1) & 3] = add2(s2[(c >> 1) & 3], p);
        pk[c >> 1] = __uint_as_float(pack2_16<KIND>(p.x, p.y));
      }
      if (j > 0) wait(XB_OD, j - 1);  // P is free once the previous product has read it
      tmem_st16(trow + XT_P + 32 * hh, pk);
      tmem_st16(trow + XT_P + 32 * hh + 16, pk + 16);
      lsum += ((s2[0].x + s2[0].y) + (s2[1].x + s2[1].y)) + ((s2[2].x + s2[2].y) + (s2[3].x + s2[3].y));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[XB_PF]);
    }
    if (nk > 0) wait(XB_OD, nk - 1);
    // the row's sum from both halves, then this half's columns of O
    float* sbuf = red + (nk & 1) * 256;  // the buffer the last tile did not use
    sbuf[hh * 128 + row] = lsum;
    pair_sync(q);
    lsum = sbuf[row] + sbuf[128 + row];
    float ov[32];
    if (nk > 0) {
      tmem_ld32(trow + XT_O + 32 * hh, ov);
      tmem_ld_wait();
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) ov[c] = 0.f;
    }
    if (S > 1) {
      block_sync();  // the block's loads and products are complete: the tiles may be overwritten
      float* part = reinterpret_cast<float*>(sm) + row * XT_PART_LD + 32 * hh;
      float* stat = reinterpret_cast<float*>(sm) + 128 * XT_PART_LD + row * 2;
#pragma unroll
      for (int c = 0; c < 32; c += 4)
        *reinterpret_cast<float4*>(part + c) = make_float4(ov[c], ov[c + 1], ov[c + 2], ov[c + 3]);
      if (hh == 0) stat[0] = m_used, stat[1] = lsum;
      __syncwarp();
      cluster_sync();
      if (row * S / 128 == rank) {
        const uint32_t as = smem_u32(stat), ap = smem_u32(part);
        m_used = -INFINITY;
        for (int b = 0; b < S; ++b) m_used = fmaxf(m_used, ld_cluster_f32(mapa_shared(as, b)));
        const float sh = shift_of(m_used);
        lsum = 0.f;
#pragma unroll
        for (int c = 0; c < 32; ++c) ov[c] = 0.f;
        for (int b = 0; b < S; ++b) {
          const uint32_t rs = mapa_shared(as, b), rp = mapa_shared(ap, b);
          const float f = ex2_approx(ld_cluster_f32(rs) - sh);
          lsum = fmaf(f, ld_cluster_f32(rs + 4), lsum);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 x = ld_cluster_f4(rp + 4 * c);
            ov[c] = fmaf(f, x.x, ov[c]), ov[c + 1] = fmaf(f, x.y, ov[c + 1]);
            ov[c + 2] = fmaf(f, x.z, ov[c + 2]), ov[c + 3] = fmaf(f, x.w, ov[c + 3]);
          }
        }
      }
      __syncwarp();
      cluster_sync();  // no block leaves while another may read its part
    }
    if (row0 + row < s.lq && (S == 1 || row * S / 128 == rank)) {
      const float inv = s.lk > 0 ? 1.0f / lsum : 0.f;  // no states: zeros
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + (long long)(s.q0 + row0 + row) * a.ldo +
                                            64 * h + 32 * hh);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float o8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o8[i] = average<KIND>(ov[8 * c + i], inv);
        dst[c] = pack8_16<KIND>(o8);
      }
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == XT_MMA_WARP) tmem_dealloc(tmem, XT_TMEM_COLS);
  if (tid == 0 && failed) atomicCAS(a.status, 0, failed);
}

template <int KIND>
static cudaError_t launch_tiles(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, XattnArgs a,
                                int n_seg, cudaStream_t st) {
  auto kern = xattn_tiles_kernel<KIND>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_once(kern, XT_SMEM, done);
  if (e != cudaSuccess) return e;
  static WideClusters seen;
  a.splits = cap_splits(a.splits, [&] { return holds_wide_cluster(kern, XT_THREADS, XT_SMEM, seen); });
  const int q_blocks = (a.max_q + 127) / 128;
  return launch_cluster(kern, dim3(n_seg * q_blocks * a.splits, a.H), XT_THREADS, XT_SMEM, a.splits, st, q, k, v, a, q_blocks);
}

cudaError_t launch_xattn_tiles(XattnArgs a, int n_seg, int max_k, bool f16, int num_sms, cudaStream_t st) {
  CUtensorMap q, k, v;
  if (!make_tmap_bf16(&q, a.q, a.Tq, 64ULL * a.H, a.ldq, 128) ||
      !make_tmap_bf16(&k, a.k, a.Tk, 64ULL * (a.H / a.G), a.ldk, 128) ||
      !make_tmap_bf16(&v, a.v, a.Tk, 64ULL * (a.H / a.G), a.ldv, 128))
    return cudaErrorInvalidValue;
  a.splits = tile_splits((double)n_seg * ((a.max_q + 127) / 128) * a.H, (max_k + 127) / 128, 12.5, num_sms);
  return f16 ? launch_tiles<KIND_F16>(q, k, v, a, n_seg, st) : launch_tiles<KIND_BF16>(q, k, v, a, n_seg, st);
}

// Attention weights of many rows: the scores of a 128-row tile of one
// (segment, selected head) from the tensor cores, twice over the states.  The
// first pass keeps each thread's running maximum and sum (its row, its half of
// every tile), joined over the two halves once at its end; the second turns
// the same scores into probabilities, staged as 32 x 32 boxes and written by
// TMA.  448 rows x 1500 states x 10 heads x 32 segments (942 MB, 144 us at the
// copy rate; twice 46 us of exponentials): 221-231 us; 64 rows a block on
// mma.sync took 402.
namespace {
constexpr int XWT_KS = 2, XWT_SK = XT_TILE, XWT_BUF = XWT_SK + XWT_KS * XT_TILE, XWT_RED = XWT_BUF + 8 * 4096;
constexpr int XWT_BARS = XWT_RED + 2 * 128 * 8;
enum { WB_Q = 0, WB_KF, WB_KE = WB_KF + XWT_KS, WB_SF = WB_KE + XWT_KS, WB_SE = WB_SF + 2, WB_DRAIN = WB_SE + 2, WB_COUNT };
constexpr int XWT_SMEM = 1024 + XWT_BARS + 8 * WB_COUNT + 16;
static_assert(2 * (XWT_SMEM + 1024) <= 228 * 1024, "two blocks per SM");
}  // namespace

template <int KIND>
__global__ void __launch_bounds__(320, 2)
    xattn_weights_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                               const __grid_constant__ CUtensorMap tm_out, const XattnArgs a, int q_blocks, int out_tma) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int failed;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + XWT_BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + WB_COUNT);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    failed = 0;
    for (int i = 0; i < WB_COUNT; ++i) mbar_init(&bar[i], i == WB_SE || i == WB_SE + 1 ? 8 : 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
  }
  if (warp == XT_MMA_WARP) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int S = a.splits, rank = blockIdx.x % S, unit = blockIdx.x / S;
  const int seg = unit / q_blocks, row0 = (unit - seg * q_blocks) * 128, sel = blockIdx.y;
  const Segment s = load_segment(a, seg, tid == 0);
  const int h = a.heads ? __ldg(a.heads + sel) : sel;
  const bool head_ok = h >= 0 && h < a.H;
  if (!head_ok && tid == 0) atomicCAS(a.status, 0, DEV_BAD_SEGMENT);
  const bool live = s.ok && head_ok && row0 < s.lq;  // the same for every block of the cluster
  // this block's tiles of columns, and how many of them hold states
  const int tiles = (a.width + 127) / 128;
  const int t0 = (int)((long long)rank * tiles / S), t1 = (int)((long long)(rank + 1) * tiles / S);
  const int nk = max(0, min(t1, (s.lk + 127) / 128) - t0);
  // Cluster barriers: the load and issue warps arrive at the first at once (it
  // only guards the softmax warps' statistics) and wait at their end.
  if (S > 1 && live && warp >= XT_TMA_WARP) cluster_arrive();

  if (live && nk > 0 && warp == XT_TMA_WARP) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&bar[WB_Q], XT_TILE);
      tma_load_2d(sm, &tm_q, &bar[WB_Q], h * 64, s.q0 + row0);
      int n = 0;
      for (; n < 2 * nk; ++n) {
        const int ks = n % XWT_KS, j = t0 + (n < nk ? n : n - nk);
        if (!mbar_wait(&bar[WB_KE + ks], ((n / XWT_KS) & 1) ^ 1, a.limit_ns, &failed, DEV_TIMEOUT_PRODUCER)) break;
        mbar_arrive_expect_tx(&bar[WB_KF + ks], XT_TILE);
        tma_load_2d(sm + XWT_SK + ks * XT_TILE, &tm_k, &bar[WB_KF + ks], h / a.G * 64, s.k0 + j * 128);
      }
      // every issued load lands before the block exits
      mbar_wait(&bar[WB_Q], 0, kDrainLimitNs, nullptr, 0);
      for (int i = max(0, n - XWT_KS); i < n; ++i)
        mbar_wait(&bar[WB_KF + i % XWT_KS], (i / XWT_KS) & 1, kDrainLimitNs, nullptr, 0);
    }
  } else if (live && nk > 0 && warp == XT_MMA_WARP) {
    const uint32_t idesc = idesc_kind_f32(KIND, 128, 128);
    const uint64_t qd = sw128_kmajor_desc(smem_u32(sm)), kd = sw128_kmajor_desc(smem_u32(sm + XWT_SK));
    auto wait = [&](int b, int n) {
      return __all_sync(0xffffffffu, mbar_wait(&bar[b], n & 1, a.limit_ns, &failed, DEV_TIMEOUT_MMA)) != 0;
    };
    bool ok = wait(WB_Q, 0);
    for (int n = 0; n < 2 * nk && ok; ++n) {
      const int b = n & 1, ks = n % XWT_KS;
      if (!(ok = wait(WB_KF + ks, n / XWT_KS) && wait(WB_SE + b, (n >> 1) ^ 1))) break;
      tc_fence_after();
      tc_scores_warp(tmem + 128 * b, qd, kd + ks * (XT_TILE >> 4), idesc);
      tc_commit_warp(&bar[WB_SF + b]);
      tc_commit_warp(&bar[WB_KE + ks]);
    }
    // all issued MMAs complete before tensor memory is released
    tc_commit_warp(&bar[WB_DRAIN]);
    mbar_wait(&bar[WB_DRAIN], 0, kDrainLimitNs, nullptr, 0);
  } else if (live && warp < XT_TMA_WARP) {
    const int q = warp & 3, hh = warp >> 2, row = 32 * q + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * q) << 16) + 64 * hh;
    float m = -INFINITY, l = 0.f, sh = 0.f, inv = 0.f;
    // After a failed wait the loops run on without waiting, so that the two
    // warps of a pair meet the same barrier.
    bool ok = true;
    auto scores = [&](int n, float* v) {
      ok = ok && mbar_wait(&bar[WB_SF + (n & 1)], (n >> 1) & 1, a.limit_ns, &failed, DEV_TIMEOUT_EPILOGUE);
      tc_fence_after();
      tmem_ld32(trow + 128 * (n & 1), v);
      tmem_ld32(trow + 128 * (n & 1) + 32, v + 32);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[WB_SE + (n & 1)]);
    };
    for (int n = 0; n < nk; ++n) {
      float v[64];
      scores(n, v);
      const int kv = s.lk - (t0 + n) * 128 - 64 * hh;  // states of this half
      if (kv < 64) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c >= kv) v[c] = -INFINITY;
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; c += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], fmaxf(v[c + 2 * i], v[c + 2 * i + 1]));
      }
      const float mn = fmaxf(m, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * kScaleLog2);
      sh = shift_of(mn);
      l *= ex2_approx(m - sh);
      m = mn;
      const float2 scale2 = make_float2(kScaleLog2, kScaleLog2), shift2 = make_float2(-sh, -sh);
      float2 s2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 x = fma2(make_float2(v[c], v[c + 1]), scale2, shift2);
        s2[(c >> 1) & 3] = add2(s2[(c >> 1) & 3], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
      }
      l += ((s2[0].x + s2[0].y) + (s2[1].x + s2[1].y)) + ((s2[2].x + s2[2].y) + (s2[3].x + s2[3].y));
    }
    // the row's maximum and sum: over both halves, and over the cluster's
    // blocks in rank order
    float2* red = reinterpret_cast<float2*>(sm + XWT_RED);
    red[hh * 128 + row] = make_float2(m, l);
    if (S > 1)
      cluster_sync();
    else
      pair_sync(q);
    if (s.lk > 0) {
      const uint32_t mine = smem_u32(&red[row]);
      float mm = -INFINITY, ll = 0.f;
      for (int i = 0; i < 2 * S; ++i) {
        const uint32_t p = mapa_shared(mine, S > 1 ? i >> 1 : 0) + (i & 1) * (128 * 8);
        mm = fmaxf(mm, S > 1 ? ld_cluster_f32(p) : red[(i & 1) * 128 + row].x);
      }
      sh = shift_of(mm);
      for (int i = 0; i < 2 * S; ++i) {
        const uint32_t p = mapa_shared(mine, S > 1 ? i >> 1 : 0) + (i & 1) * (128 * 8);
        const float2 x = S > 1 ? make_float2(ld_cluster_f32(p), ld_cluster_f32(p + 4)) : red[(i & 1) * 128 + row];
        ll = fmaf(x.y, ex2_approx(x.x - sh), ll);
      }
      inv = 1.0f / ll;
    }
    if (S > 1) cluster_arrive();  // the others' statistics have been read
    uint8_t* buf = sm + XWT_BUF + warp * 4096;
    const int rows = s.lq - row0 - 32 * q;  // valid rows of this warp, if fewer than 32
    const long long orow = (long long)sel * a.Tq + s.q0 + row0 + 32 * q;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.out) & 15) | (a.ldo & 3)) == 0;
    for (int j = t0; j < t1 && j * 128 + 64 * hh < a.width && rows > 0; ++j) {
      float v[64];
      if (j - t0 < nk) {
        scores(nk + j - t0, v);
      } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] = 0.f;  // columns past the states: zeros below
      }
      const int kv = s.lk - j * 128 - 64 * hh;
      const float2 scale2 = make_float2(kScaleLog2, kScaleLog2), shift2 = make_float2(-sh, -sh), inv2 = make_float2(inv, inv);
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 x = fma2(make_float2(v[c], v[c + 1]), scale2, shift2);
        const float2 p = mul2(make_float2(ex2_approx(x.x), ex2_approx(x.y)), inv2);
        v[c] = p.x, v[c + 1] = p.y;
      }
      if (kv < 64) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c >= kv) v[c] = 0.f;
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int x0 = j * 128 + 64 * hh + 32 * b;
        if (x0 >= a.width) break;
        if (lane == 0) bulk_wait_read0();  // the box stored last has been read
        __syncwarp();
        float4* dst = reinterpret_cast<float4*>(buf + lane * 128);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          dst[k ^ (lane & 7)] = make_float4(v[32 * b + 4 * k], v[32 * b + 4 * k + 1], v[32 * b + 4 * k + 2], v[32 * b + 4 * k + 3]);
        // (a store clips a box at the width rounded up to whole 16 bytes)
        if (out_tma && rows >= 32 && (x0 + 32 <= a.width || a.width % 4 == 0)) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_out, buf, x0, static_cast<int>(orow));
            bulk_commit();
          }
        } else {
          // rows of the next segment follow inside the box, or rows or the
          // width are not whole 16 bytes: eight lanes a row
          __syncwarp();
#pragma unroll 1
          for (int r = lane >> 3; r < min(32, rows); r += 4) {
            const float4 f = reinterpret_cast<const float4*>(buf + r * 128)[(lane & 7) ^ (r & 7)];
            const int x = x0 + 4 * (lane & 7);
            float* o = reinterpret_cast<float*>(a.out) + (orow + r) * a.ldo + x;
            if (vec && x + 4 <= a.width) {
              *reinterpret_cast<float4*>(o) = f;
            } else {
              if (x < a.width) o[0] = f.x;
              if (x + 1 < a.width) o[1] = f.y;
              if (x + 2 < a.width) o[2] = f.z;
              if (x + 3 < a.width) o[3] = f.w;
            }
          }
          __syncwarp();
        }
      }
    }
    // a warp without rows still gives back the scores of the second pass
    if (rows <= 0) {
      for (int j = 0; j < nk; ++j) {
        ok = ok && mbar_wait(&bar[WB_SF + ((nk + j) & 1)], ((nk + j) >> 1) & 1, a.limit_ns, &failed, DEV_TIMEOUT_EPILOGUE);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[WB_SE + ((nk + j) & 1)]);
      }
    } else if (nk > 0 && (t0 + nk - 1) * 128 + 64 * hh >= a.width) {
      // (the last tile's second half lies past the width)
      ok = ok && mbar_wait(&bar[WB_SF + ((2 * nk - 1) & 1)], ((2 * nk - 1) >> 1) & 1, a.limit_ns, &failed, DEV_TIMEOUT_EPILOGUE);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[WB_SE + ((2 * nk - 1) & 1)]);
    }
    if (lane == 0) bulk_wait0();
    __syncwarp();
    if (S > 1) cluster_wait();  // no block leaves while another may read its statistics
  }
  if (S > 1 && live && warp >= XT_TMA_WARP) {
    __syncwarp();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == XT_MMA_WARP) tmem_dealloc(tmem, 256);
  if (tid == 0 && failed) atomicCAS(a.status, 0, failed);
}

cudaError_t launch_xattn_weights_tiles(XattnArgs a, int n_seg, int n_sel, bool f16, int num_sms, cudaStream_t st) {
  CUtensorMap q, k, o;
  if (!make_tmap_bf16(&q, a.q, a.Tq, 64ULL * a.H, a.ldq, 128) ||
      !make_tmap_bf16(&k, a.k, a.Tk, 64ULL * (a.H / a.G), a.ldk, 128))
    return cudaErrorInvalidValue;
  const bool tma = n_sel * a.Tq < (1LL << 31) && make_tmap_out(&o, a.out, n_sel * a.Tq, a.width, a.ldo, true);
  if (!tma) o = k;
  const int q_blocks = (a.max_q + 127) / 128;
  // as for the attention, with two passes over each tile
  a.splits = tile_splits((double)n_seg * q_blocks * n_sel, (a.width + 127) / 128, 25.0, num_sms);
  auto kern = f16 ? xattn_weights_tiles_kernel<KIND_F16> : xattn_weights_tiles_kernel<KIND_BF16>;
  static std::atomic<unsigned long long> done[2] = {{0}, {0}};
  const cudaError_t e = set_smem_once(kern, XWT_SMEM, done[f16]);
  if (e != cudaSuccess) return e;
  static WideClusters seen[2];
  a.splits = cap_splits(a.splits, [&] { return holds_wide_cluster(kern, 320, XWT_SMEM, seen[f16]); });
  return launch_cluster(kern, dim3(n_seg * q_blocks * a.splits, n_sel), 320, XWT_SMEM, a.splits, st, q, k, o, a, q_blocks, (int)tma);
}

}  // namespace asr
