// Cross attention of many rows on the tcgen05 tensor cores.
//
// One block takes NT tiles of 128 rows of one (segment, head) over the
// segment's states in tiles of 128:
//   warp 4 NT      TMA: the query tiles once, then K_j and V_j into rings;
//   warp 4 NT + 1  MMA: S_t = Q_t K_j^T (128 x 128 x 64), then
//                  O_t += P_t V_j (128 x 64 x 128) with P_t read from tensor
//                  memory;
//   warps 4 t .. 4 t + 3  softmax of tile t, one row per thread: the row's 128
//                  scores are read into registers at once, so S_t is free for
//                  the next tile's product while the exponentials run.
// Tensor memory per tile: S 128, O 64, P 64 columns, none of them shared, so
// the products of tile j + 1 overlap the softmax of tile j.  With NT = 2 the
// two tiles share every K_j and V_j, and one tile's exponentials run while the
// other waits for the tensor cores.
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

template <int NT_>
struct XtShape {
  static constexpr int NT = NT_;
  static constexpr int STAGES = NT == 2 ? 4 : 2;  // K and V tiles in flight (one block per SM, or two)
  static constexpr int THREADS = 32 * (4 * NT + 2);
  static constexpr int TMA_WARP = 4 * NT, MMA_WARP = 4 * NT + 1;
  static constexpr int TILE = 16384;
  static constexpr int SQ = 0, SK = NT * TILE, SV = SK + STAGES * TILE, BARS = SV + STAGES * TILE;
  // barriers: Q, K full / empty, V full / empty, and per tile S full, S free, P full, PV done; drain
  static constexpr int B_Q = 0, B_KF = 1, B_KE = B_KF + STAGES, B_VF = B_KE + STAGES, B_VE = B_VF + STAGES,
                       B_SF = B_VE + STAGES, B_SE = B_SF + NT, B_PF = B_SE + NT, B_OD = B_PF + NT, B_DRAIN = B_OD + NT,
                       B_COUNT = B_DRAIN + 1;
  static constexpr int SMEM = 1024 + BARS + 8 * B_COUNT + 16;
  // the parts of a split row reuse the tiles: 64 floats of O (row padded to 68), then maximum and sum
  static constexpr int PART_LD = 68;
  static_assert(NT * 128 * (PART_LD + 2) * 4 <= BARS, "parts fit in the tiles");
  static constexpr int TMEM_COLS = 256 * NT;
  static constexpr int S_COL = 0, P_COL = 128, O_COL = 192;  // within a tile's 256 columns
};

// D[tmem] (+)= A[tmem] * B[smem]: A's rows are lanes, two 16-bit elements of K per column.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

}  // namespace

template <int KIND, int NT>
__global__ void __launch_bounds__(XtShape<NT>::THREADS, 3 - NT)
    xattn_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const XattnArgs a, int q_blocks) {
  using X = XtShape<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int failed;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + X::BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + X::B_COUNT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    failed = 0;
    for (int i = 0; i < X::B_COUNT; ++i) mbar_init(&bar[i], i >= X::B_SE && i < X::B_OD ? 4 : 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == X::MMA_WARP) {
    tmem_alloc(tmem_slot, X::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const int S = a.splits, rank = blockIdx.x % S, unit = blockIdx.x / S;
  const int seg = unit / q_blocks, row0 = (unit - seg * q_blocks) * (128 * NT), h = blockIdx.y, kvh = h / a.G;
  const Segment s = load_segment(a, seg, tid == 0);
  const bool live = s.ok && row0 < s.lq;  // the same for every block of the cluster
  const int nt = NT == 2 && row0 + 128 < s.lq ? 2 : 1;
  // this block's tiles of states
  const int tiles = (s.lk + 127) / 128, t0 = (int)((long long)rank * tiles / S), t1 = (int)((long long)(rank + 1) * tiles / S);
  const int nk = t1 - t0;
  float m_used = -INFINITY, lsum = 0.f;  // softmax threads: of their row

  if (live && nk > 0) {
    if (warp == X::TMA_WARP) {
      if (lane == 0) {
        const int k0 = s.k0 + t0 * 128;
        mbar_arrive_expect_tx(&bar[X::B_Q], nt * X::TILE);
        for (int t = 0; t < nt; ++t) tma_load_2d(sm + X::SQ + t * X::TILE, &tm_q, &bar[X::B_Q], h * 64, s.q0 + row0 + 128 * t);
        int nkl = 0, nvl = 0;
        for (int j = 0; j < nk; ++j) {
          const int st = j % X::STAGES;
          const uint32_t ph = ((j / X::STAGES) & 1) ^ 1;
          if (!mbar_wait_bounded(&bar[X::B_KE + st], ph, a.limit_ns, &failed, DEV_TIMEOUT_PRODUCER)) break;
          mbar_arrive_expect_tx(&bar[X::B_KF + st], X::TILE);
          tma_load_2d(sm + X::SK + st * X::TILE, &tm_k, &bar[X::B_KF + st], kvh * 64, k0 + j * 128);
          ++nkl;
          if (!mbar_wait_bounded(&bar[X::B_VE + st], ph, a.limit_ns, &failed, DEV_TIMEOUT_PRODUCER)) break;
          mbar_arrive_expect_tx(&bar[X::B_VF + st], X::TILE);
          tma_load_2d(sm + X::SV + st * X::TILE, &tm_v, &bar[X::B_VF + st], kvh * 64, k0 + j * 128);
          ++nvl;
        }
        // every issued load lands before the shared memory is reused or left
        mbar_wait_bounded(&bar[X::B_Q], 0, kDrainLimitNs, nullptr, 0);
        for (int j = max(0, nkl - X::STAGES); j < nkl; ++j)
          mbar_wait_bounded(&bar[X::B_KF + j % X::STAGES], (j / X::STAGES) & 1, kDrainLimitNs, nullptr, 0);
        for (int j = max(0, nvl - X::STAGES); j < nvl; ++j)
          mbar_wait_bounded(&bar[X::B_VF + j % X::STAGES], (j / X::STAGES) & 1, kDrainLimitNs, nullptr, 0);
      }
    } else if (warp == X::MMA_WARP) {
      if (lane == 0) {
        const uint32_t idesc_s = idesc_kind_f32(KIND, 128, 128);
        const uint32_t idesc_o = idesc_kind_f32(KIND, 128, 64) | (1u << 16);  // B = V, MN-major
        auto wait = [&](int b, int n) { return mbar_wait_bounded(&bar[b], n & 1, a.limit_ns, &failed, DEV_TIMEOUT_MMA); };
        auto issue_s = [&](int t, int j) {
          const uint64_t qd = sw128_kmajor_desc(smem_u32(sm + X::SQ + t * X::TILE));
          const uint64_t kd = sw128_kmajor_desc(smem_u32(sm + X::SK + (j % X::STAGES) * X::TILE));
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k) tc_mma_bf16(tmem + 256 * t + X::S_COL, qd + 2 * k, kd + 2 * k, idesc_s, k > 0);
          tc_commit(&bar[X::B_SF + t]);
          if (t == nt - 1) tc_commit(&bar[X::B_KE + j % X::STAGES]);
        };
        bool ok = wait(X::B_Q, 0) && wait(X::B_KF, 0);
        for (int t = 0; t < nt && ok; ++t) issue_s(t, 0);
        for (int j = 0; j < nk && ok; ++j) {
          for (int t = 0; t < nt && ok; ++t) {
            if (j + 1 < nk) {
              // the next scores, once the softmax holds these in registers
              const int st = (j + 1) % X::STAGES;
              if (!(ok = wait(X::B_KF + st, (j + 1) / X::STAGES) && wait(X::B_SE + t, j))) break;
              issue_s(t, j + 1);
            }
            const int st = j % X::STAGES;
            if (!(ok = wait(X::B_PF + t, j) && wait(X::B_VF + st, j / X::STAGES))) break;
            tc_fence_after();
            const uint64_t vd = sw128_mnmajor_desc(smem_u32(sm + X::SV + st * X::TILE));
#pragma unroll
            for (int k = 0; k < 8; ++k)
              tc_mma_ts(tmem + 256 * t + X::O_COL, tmem + 256 * t + X::P_COL + 8 * k, vd + (uint64_t)(k * 128), idesc_o,
                        (j > 0 || k > 0) ? 1u : 0u);
            tc_commit(&bar[X::B_OD + t]);
            if (t == nt - 1) tc_commit(&bar[X::B_VE + st]);
          }
        }
        // all issued MMAs complete before tensor or shared memory is released
        tc_commit(&bar[X::B_DRAIN]);
        mbar_wait_bounded(&bar[X::B_DRAIN], 0, kDrainLimitNs, nullptr, 0);
      }
    } else if (warp < 4 * nt) {
      const int t = warp >> 2, q = warp & 3;
      const uint32_t trow = tmem + 256 * t + (static_cast<uint32_t>(32 * q) << 16);
      auto wait = [&](int b, int n) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(&bar[b], n & 1, a.limit_ns, &failed, DEV_TIMEOUT_EPILOGUE)) != 0;
      };
      bool ok = true;
      for (int j = 0; j < nk; ++j) {
        if (!(ok = wait(X::B_SF + t, j))) break;
        tc_fence_after();
        float sv[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32(trow + X::S_COL + c, sv + c);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[X::B_SE + t]);
        const int kv = s.lk - (t0 + j) * 128;  // states of this tile, if fewer than 128
        if (kv < 128) {
          // scores past the end never count, and values past it, which may be
          // anything (another segment's), become zeros: 0 * NaN would stay NaN
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= kv) sv[c] = -INFINITY;
          if (t == 0) {
            const int st = j % X::STAGES;
            if (!(ok = wait(X::B_VF + st, j / X::STAGES))) break;
            uint4* rows = reinterpret_cast<uint4*>(sm + X::SV + st * X::TILE);
            for (int i = kv * 8 + (tid & 127); i < 1024; i += 128) rows[i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], fmaxf(sv[c + 2 * i], sv[c + 2 * i + 1]));
        }
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * kScaleLog2;
        const bool grow = mt > m_used + kRescaleLog2;
        const float m_old = m_used;
        if (grow) m_used = mt;
        const float sh = shift_of(m_used);
        // P_t and O_t are free once the previous product is complete
        if (j > 0 && !(ok = wait(X::B_OD + t, j - 1))) break;
        tc_fence_after();
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
          const float corr = grow ? ex2_approx(m_old - sh) : 1.0f;
          lsum *= corr;
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            float ov[16];
            tmem_ld16(trow + X::O_COL + c, ov);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) ov[i] *= corr;
            tmem_st16(trow + X::O_COL + c, ov);
          }
        }
        const float2 scale2 = make_float2(kScaleLog2, kScaleLog2), shift2 = make_float2(-sh, -sh);
        float2 s2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          float pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 x = fma2(make_float2(sv[c + i], sv[c + i + 1]), scale2, shift2);
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            s2[(i >> 1) & 3] = add2(s2[(i >> 1) & 3], p);
            pk[i >> 1] = __uint_as_float(pack2_16<KIND>(p.x, p.y));
          }
          tmem_st16(trow + X::P_COL + c / 2, pk);
        }
        lsum += ((s2[0].x + s2[0].y) + (s2[1].x + s2[1].y)) + ((s2[2].x + s2[2].y) + (s2[3].x + s2[3].y));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[X::B_PF + t]);
      }
      if (ok) wait(X::B_OD + t, nk - 1);
      tc_fence_after();
    }
  }

  const int t = warp >> 2, row = tid & 127;
  const bool mine = live && warp < 4 * nt;
  float ov[64];
  if (mine) {
    if (nk > 0) {
      const uint32_t trow = tmem + 256 * t + X::O_COL + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
#pragma unroll
      for (int c = 0; c < 64; c += 32) tmem_ld32(trow + c, ov + c);
      tmem_ld_wait();
    } else {
#pragma unroll
      for (int c = 0; c < 64; ++c) ov[c] = 0.f;
    }
  }
  if (S > 1 && live) {
    __syncthreads();  // the block's loads and products are complete: the tiles may be overwritten
    float* part = reinterpret_cast<float*>(sm) + (t * 128 + row) * X::PART_LD;
    float* stat = reinterpret_cast<float*>(sm) + NT * 128 * X::PART_LD + (t * 128 + row) * 2;
    if (mine) {
#pragma unroll
      for (int c = 0; c < 64; c += 4) *reinterpret_cast<float4*>(part + c) = make_float4(ov[c], ov[c + 1], ov[c + 2], ov[c + 3]);
      stat[0] = m_used;
      stat[1] = lsum;
    }
    __syncwarp();
    cluster_sync();
    if (mine && row * S / 128 == rank) {
      const uint32_t as = smem_u32(stat), ap = smem_u32(part);
      m_used = -INFINITY;
      for (int b = 0; b < S; ++b) m_used = fmaxf(m_used, ld_cluster_f32(mapa_shared(as, b)));
      const float sh = shift_of(m_used);
      lsum = 0.f;
#pragma unroll
      for (int c = 0; c < 64; ++c) ov[c] = 0.f;
      for (int b = 0; b < S; ++b) {
        const uint32_t rs = mapa_shared(as, b), rp = mapa_shared(ap, b);
        const float f = ex2_approx(ld_cluster_f32(rs) - sh);
        lsum = fmaf(f, ld_cluster_f32(rs + 4), lsum);
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float4 x = ld_cluster_f4(rp + 4 * c);
          ov[c] = fmaf(f, x.x, ov[c]), ov[c + 1] = fmaf(f, x.y, ov[c + 1]);
          ov[c + 2] = fmaf(f, x.z, ov[c + 2]), ov[c + 3] = fmaf(f, x.w, ov[c + 3]);
        }
      }
    }
    __syncwarp();
    cluster_sync();  // no block leaves while another may read its part
  }
  if (mine && row0 + 128 * t + row < s.lq && (S == 1 || row * S / 128 == rank)) {
    const float inv = s.lk > 0 ? 1.0f / lsum : 0.f;  // no states: zeros
    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) +
                                          (long long)(s.q0 + row0 + 128 * t + row) * a.ldo + 64 * h);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float o8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o8[i] = ov[8 * c + i] * inv;
      dst[c] = pack8_16<KIND>(o8);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == X::MMA_WARP) tmem_dealloc(tmem, X::TMEM_COLS);
  if (tid == 0 && failed) atomicCAS(a.status, 0, failed);
}

template <int KIND, int NT>
static cudaError_t launch_tiles(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const XattnArgs& a,
                                int n_seg, cudaStream_t st) {
  using X = XtShape<NT>;
  auto kern = xattn_tiles_kernel<KIND, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, X::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  const int q_blocks = (a.max_q + 128 * NT - 1) / (128 * NT);
  return launch_split(kern, dim3(n_seg * q_blocks * a.splits, a.H), X::THREADS, X::SMEM, a.splits, st, q, k, v, a, q_blocks);
}

cudaError_t launch_xattn_tiles(XattnArgs a, int n_seg, int max_k, bool f16, int num_sms, cudaStream_t st) {
  CUtensorMap q, k, v;
  if (!make_tmap_bf16(&q, a.q, a.Tq, 64ULL * a.H, a.ldq, 128) ||
      !make_tmap_bf16(&k, a.k, a.Tk, 64ULL * (a.H / a.G), a.ldk, 128) ||
      !make_tmap_bf16(&v, a.v, a.Tk, 64ULL * (a.H / a.G), a.ldv, 128))
    return cudaErrorInvalidValue;
  const bool two = a.max_q > 128;
  const int rows = two ? 256 : 128;
  const long long blocks = (long long)n_seg * ((a.max_q + rows - 1) / rows) * a.H;
  a.splits = pick_splits(blocks, max_k, 256, num_sms);
  if (two) return f16 ? launch_tiles<KIND_F16, 2>(q, k, v, a, n_seg, st) : launch_tiles<KIND_BF16, 2>(q, k, v, a, n_seg, st);
  return f16 ? launch_tiles<KIND_F16, 1>(q, k, v, a, n_seg, st) : launch_tiles<KIND_BF16, 1>(q, k, v, a, n_seg, st);
}

}  // namespace asr
