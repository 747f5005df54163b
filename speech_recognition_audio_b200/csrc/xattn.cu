// Cross attention: a decoder's tokens over the encoder states of their clip
// ("CrisperWhisper -> ONNX (with cross-attentions)", What this exports
// instead: whisper-small decoder; Results: a (1, 12, 1, 1500) attention
// tensor per token), and the attention weights themselves.
//
//   s_ij = q_i . k_j / 8,  p_ij = exp(s_ij - m_i) / sum_j exp(s_ij - m_i),
//   out_i = sum_j p_ij v_j,  weights_ij = p_ij   (m_i = max_j s_ij)
//
// over the states j of row i's segment; a segment without states gives zeros.
// Heads are 64 wide; G = H / Hkv query heads share one key / value head.
//
// Few rows: a tile of 8 or 16 rows (tokens x shared heads) per block, where the
// time is that of reading the states once.  The keys are split over the
// warps of a block and the blocks of a cluster, each warp keeping a running
// maximum and sum of its own; the parts are joined in a fixed order through
// shared and distributed shared memory.  Both products run transposed, states
// (or value elements) along the 16 rows of mma.sync and 8 query rows along its
// columns: S^T = K Q^T, O^T += V^T P^T, with P^T turned by movmatrix.  Keys and
// values go from global memory straight into operand registers (no shared
// memory on the way): a contraction may visit its terms in any order, so lane
// (g, t) of the fragment layout takes whole 16-byte pieces of a key row and
// the query fragments follow the same order, and the values' elements are
// permuted the same way.  mma.sync rather than tcgen05: a 128-row tile would
// be all but empty.
#include "xattn.cuh"

namespace asr {

namespace {

template <int KIND>
__device__ __forceinline__ void mma16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (KIND == KIND_F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld16(const uint16_t* p, bool valid) {
  return valid ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}
// Transpose of an 8 x 8 matrix of 16-bit elements, a row's pair per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Query fragments of 16 rows (tokens row0 ..) of head h: lane (g, t) holds, of
// rows g and g + 8, elements 8 t .. 8 t + 7 and 32 + 8 t .. 32 + 8 t + 7, i.e.
// k step s is elements 32 (s / 2) + 8 t + 4 (s % 2) + 0..3.
__device__ __forceinline__ void load_q16(const XattnArgs& a, const Segment& s, int row0, int h, int lane,
                                         uint32_t (*qf)[4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int tok = row0 + g + 8 * hh;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q) + (long long)(s.q0 + tok) * a.ldq + 64 * h + 8 * t;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 u = ld16(p + 32 * c, tok < s.lq);
      qf[2 * c][hh] = u.x;
      qf[2 * c][2 + hh] = u.y;
      qf[2 * c + 1][hh] = u.z;
      qf[2 * c + 1][2 + hh] = u.w;
    }
  }
}

// Scores of 16 rows and the 8 keys whose pieces (lo, hi) the lanes hold.
template <int KIND>
__device__ __forceinline__ void scores8(float* c, const uint32_t (*qf)[4], const uint4& lo, const uint4& hi) {
  c[0] = c[1] = c[2] = c[3] = 0.f;
  mma16<KIND>(c, qf[0], lo.x, lo.y);
  mma16<KIND>(c, qf[1], lo.z, lo.w);
  mma16<KIND>(c, qf[2], hi.x, hi.y);
  mma16<KIND>(c, qf[3], hi.z, hi.w);
}

constexpr int XS_KEYS = 32;  // keys of a warp's step

}  // namespace

template <int KIND, int NB, int W>
__global__ void __launch_bounds__(32 * W, NB == 1 ? 16 / W : W == 4 ? 3 : 1) xattn_rows_kernel(const XattnArgs a) {
  constexpr int ROWS = 8 * NB;
  __shared__ __align__(16) float so[W][ROWS][68];  // rows padded against bank conflicts
  __shared__ float sm[W][ROWS], sl[W][ROWS];
  __shared__ float cm[ROWS], cl[ROWS];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int S = a.splits, seg = blockIdx.x / S, rank = blockIdx.x - seg * S;
  const int row0 = blockIdx.y * ROWS, kvh = blockIdx.z, G = a.G;
  const Segment s = load_segment(a, seg, tid == 0);
  if (!s.ok || row0 >= s.lq * G) return;  // the same for every block of the cluster

  // Row r of the tile: token r / G, head kvh G + r % G.  Lane (g, t) holds, of
  // row g of each 8, elements 8 t .. 8 t + 7 and 32 + 8 t .. 32 + 8 t + 7.
  uint4 qf[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = row0 + 8 * nb + g, tok = r / G, h = kvh * G + (r - tok * G);
    const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q) + (long long)(s.q0 + tok) * a.ldq + 64 * h + 8 * t;
    qf[nb][0] = ld16(p, tok < s.lq);
    qf[nb][1] = ld16(p + 32, tok < s.lq);
  }
  // this block's keys, in whole steps of a warp
  const int steps = (s.lk + XS_KEYS - 1) / XS_KEYS;
  const int lo = rank * steps / S * XS_KEYS, hi = min((rank + 1) * steps / S * XS_KEYS, s.lk);
  const uint16_t* kp = reinterpret_cast<const uint16_t*>(a.k) + (long long)s.k0 * a.ldk + 64 * kvh + 8 * t;
  const uint16_t* vp = reinterpret_cast<const uint16_t*>(a.v) + (long long)s.k0 * a.ldv + 64 * kvh + 8 * g;
  // o[nb][d]: elements 8 g + 2 d and 8 g + 2 d + 1 of rows 2 t and 2 t + 1
  float o[NB][4][4], m[NB][2], l[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int d = 0; d < 4; ++d) o[nb][d][0] = o[nb][d][1] = o[nb][d][2] = o[nb][d][3] = 0.f;
    m[nb][0] = m[nb][1] = -INFINITY;
    l[nb][0] = l[nb][1] = 0.f;
  }
  for (int j0 = lo + warp * XS_KEYS; j0 < hi; j0 += W * XS_KEYS) {
    uint4 kf[4][2], vf[2][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + 8 * u + g;
#pragma unroll
      for (int c = 0; c < 2; ++c) kf[u][c] = ld16(kp + (long long)j * a.ldk + 32 * c, j < hi);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + 16 * u + 2 * t + (i & 1) + 8 * (i >> 1);
        vf[u][i] = ld16(vp + (long long)j * a.ldv, j < hi);
      }
    uint32_t pf[NB][2][2];  // P^T: [16 states][half]
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      // c[w]: states j0 + 16 w + g (0, 1) and + 8 (2, 3), rows 2 t and 2 t + 1
      float c[2][4];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        c[w][0] = c[w][1] = c[w][2] = c[w][3] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 x = kf[2 * w][i], y = kf[2 * w + 1][i], b = qf[nb][i];
          const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
          mma16<KIND>(c[w], a0, b.x, b.y);
          mma16<KIND>(c[w], a1, b.z, b.w);
        }
      }
      // keys past the end never count, whatever the arrays hold there
      if (j0 + XS_KEYS > hi) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j0 + 16 * w + 8 * (i >> 1) + g >= hi) c[w][i] = -INFINITY;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(fmaxf(c[0][r], c[0][2 + r]), fmaxf(c[1][r], c[1][2 + r]));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        mx = fmaxf(m[nb][r], mx * kScaleLog2);
        const float sh = shift_of(mx), corr = ex2_approx(m[nb][r] - sh);
        m[nb][r] = mx;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = r; i < 4; i += 2) {
            c[w][i] = ex2_approx(fmaf(c[w][i], kScaleLog2, -sh));
            sum += c[w][i];
          }
        l[nb][r] = l[nb][r] * corr + sum;  // of this lane's states
#pragma unroll
        for (int d = 0; d < 4; ++d) o[nb][d][r] *= corr, o[nb][d][2 + r] *= corr;
      }
      // probabilities rounded to the values' type, the operand type of the product
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        pf[nb][w][0] = transpose8(pack2_16<KIND>(c[w][0], c[w][1]));
        pf[nb][w][1] = transpose8(pack2_16<KIND>(c[w][2], c[w][3]));
      }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vf[w][0]);
      const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vf[w][1]);
      const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vf[w][2]);
      const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vf[w][3]);
      // row g of product d is element 8 g + 2 d, row g + 8 element 8 g + 2 d + 1
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t va[4] = {__byte_perm(v0[d], v1[d], 0x5410), __byte_perm(v0[d], v1[d], 0x7632),
                                __byte_perm(v2[d], v3[d], 0x5410), __byte_perm(v2[d], v3[d], 0x7632)};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma16<KIND>(o[nb][d], va, pf[nb][w][0], pf[nb][w][1]);
      }
    }
  }
  // this warp's part
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 8 * nb + 2 * t + r;
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], x);
      if (g == 0) sm[warp][row] = m[nb][r], sl[warp][row] = l[nb][r];
      float* dst = &so[warp][row][8 * g];
      *reinterpret_cast<float4*>(dst) = make_float4(o[nb][0][r], o[nb][0][2 + r], o[nb][1][r], o[nb][1][2 + r]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(o[nb][2][r], o[nb][2][2 + r], o[nb][3][r], o[nb][3][2 + r]);
    }
  __syncthreads();
  // join the warps: thread (row, 8 elements); the result replaces warp 0's part
  float acc[8], mm = -INFINITY, ll = 0.f;
  if (tid < 8 * ROWS) {
    const int row = tid >> 3, c8 = 8 * (tid & 7);
#pragma unroll
    for (int w = 0; w < W; ++w) mm = fmaxf(mm, sm[w][row]);
    const float sh = shift_of(mm);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = ex2_approx(sm[w][row] - sh);
      ll += f * sl[w][row];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(f, so[w][row][c8 + i], acc[i]);
    }
    if (S > 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) so[0][row][c8 + i] = acc[i];  // only this thread reads or writes these
      if ((tid & 7) == 0) cm[row] = mm, cl[row] = ll;
    }
  }
  const int mine = S > 1 ? tid * S + rank : tid;  // the (row, 8 elements) piece this thread finishes
  if (S > 1) {
    __syncwarp();
    cluster_sync();
    if (mine < 8 * ROWS) {
      const int r = mine >> 3, e = 8 * (mine & 7);
      const uint32_t am = smem_u32(&cm[r]), al = smem_u32(&cl[r]), ao = smem_u32(&so[0][r][e]);
      mm = -INFINITY;
      ll = 0.f;
      for (int b = 0; b < S; ++b) mm = fmaxf(mm, ld_cluster_f32(mapa_shared(am, b)));
      const float sh = shift_of(mm);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      for (int b = 0; b < S; ++b) {
        const float f = ex2_approx(ld_cluster_f32(mapa_shared(am, b)) - sh);
        ll += f * ld_cluster_f32(mapa_shared(al, b));
        const uint32_t ro = mapa_shared(ao, b);
        const float4 x = ld_cluster_f4(ro), y = ld_cluster_f4(ro + 16);
        acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]), acc[2] = fmaf(f, x.z, acc[2]);
        acc[3] = fmaf(f, x.w, acc[3]), acc[4] = fmaf(f, y.x, acc[4]), acc[5] = fmaf(f, y.y, acc[5]);
        acc[6] = fmaf(f, y.z, acc[6]), acc[7] = fmaf(f, y.w, acc[7]);
      }
    }
    __syncwarp();
    cluster_sync();  // no block leaves while another may read its part
  }
  if (mine < 8 * ROWS) {
    const int rr = row0 + (mine >> 3), e = 8 * (mine & 7);
    const int tok = rr / G, h = kvh * G + (rr - tok * G);
    if (tok < s.lq) {
      const float inv = s.lk > 0 ? 1.0f / ll : 0.f;  // no states: zeros
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = average<KIND>(acc[i], inv);
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + (long long)(s.q0 + tok) * a.ldo + 64 * h + e) =
          pack8_16<KIND>(acc);
    }
  }
}

// Attention weights of one selected head, 16 rows per block (few rows; many go
// to the tensor-core tiles).  Two passes over the keys (the second finds them
// in L2): running maximum and sum, joined over warps and the blocks of the
// cluster; then the scores again, written as probabilities in 32 bits.  A
// row's 8 keys of a product are one 32-byte sector of the output.
constexpr int XW_WARPS = 8, XW_KEYS = 32;

template <int KIND>
__global__ void __launch_bounds__(32 * XW_WARPS, 2) xattn_weights_kernel(const XattnArgs a) {
  __shared__ float sm[XW_WARPS][16], sl[XW_WARPS][16];
  __shared__ float cm[16], cl[16];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int S = a.splits, seg = blockIdx.x / S, rank = blockIdx.x - seg * S;
  const int row0 = blockIdx.y * 16;
  const Segment s = load_segment(a, seg, tid == 0);
  const int h = a.heads ? __ldg(a.heads + blockIdx.z) : blockIdx.z;
  const bool head_ok = h >= 0 && h < a.H;
  if (!head_ok && tid == 0) atomicCAS(a.status, 0, DEV_BAD_SEGMENT);
  if (!s.ok || !head_ok || row0 >= s.lq) return;  // the same for every block of the cluster

  uint32_t qf[4][4];
  load_q16(a, s, row0, h, lane, qf);
  const uint16_t* kp = reinterpret_cast<const uint16_t*>(a.k) + (long long)s.k0 * a.ldk + 64 * (h / a.G) + 8 * t;
  const int steps = (a.width + XW_KEYS - 1) / XW_KEYS;
  const int lo = rank * steps / S * XW_KEYS, end = min((rank + 1) * steps / S * XW_KEYS, a.width);
  const int hi = min(end, s.lk);

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  auto load_k = [&](int j0, uint4 (*kf)[2]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + 8 * u + g;
#pragma unroll
      for (int c = 0; c < 2; ++c) kf[u][c] = ld16(kp + (long long)j * a.ldk + 32 * c, j < hi);
    }
  };
  constexpr int STEP = XW_WARPS * XW_KEYS;
  uint4 kf[4][2];
  load_k(lo + warp * XW_KEYS, kf);
  for (int j0 = lo + warp * XW_KEYS; j0 < hi; j0 += STEP) {
    uint4 kn[4][2];
    load_k(j0 + STEP, kn);
    {
      float c[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) scores8<KIND>(c[u], qf, kf[u][0], kf[u][1]);
      if (j0 + XW_KEYS > hi) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j0 + 8 * u + 2 * t + (i & 1) >= hi) c[u][i] = -INFINITY;
      }
      // per lane: its four lanes of a row are joined once at the end
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float mx = fmaxf(c[0][2 * hh], c[0][2 * hh + 1]);
#pragma unroll
        for (int u = 1; u < 4; ++u) mx = fmaxf(mx, fmaxf(c[u][2 * hh], c[u][2 * hh + 1]));
        const float mn = fmaxf(m[hh], mx * kScaleLog2), sh = shift_of(mn);
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 2 * hh; i < 2 * hh + 2; ++i) sum += ex2_approx(fmaf(c[u][i], kScaleLog2, -sh));
        l[hh] = l[hh] * ex2_approx(m[hh] - sh) + sum;
        m[hh] = mn;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) kf[u][0] = kn[u][0], kf[u][1] = kn[u][1];
  }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float mm = m[hh];
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 2));
      float ll = l[hh] * ex2_approx(m[hh] - shift_of(mm));
      ll += __shfl_xor_sync(0xffffffffu, ll, 1);
      ll += __shfl_xor_sync(0xffffffffu, ll, 2);
      if (t == 0) sm[warp][g + 8 * hh] = mm, sl[warp][g + 8 * hh] = ll;
    }
  __syncthreads();
  if (tid < 16) {
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < XW_WARPS; ++w) mm = fmaxf(mm, sm[w][tid]);
    const float sh = shift_of(mm);
#pragma unroll
    for (int w = 0; w < XW_WARPS; ++w) ll += ex2_approx(sm[w][tid] - sh) * sl[w][tid];
    cm[tid] = mm, cl[tid] = ll;
  }
  if (S > 1) {
    __syncwarp();
    cluster_sync();
    float mm = -INFINITY, ll = 0.f;
    if (tid < 16) {
      for (int b = 0; b < S; ++b) mm = fmaxf(mm, ld_cluster_f32(mapa_shared(smem_u32(&cm[tid]), b)));
      const float sh = shift_of(mm);
      for (int b = 0; b < S; ++b)
        ll += ex2_approx(ld_cluster_f32(mapa_shared(smem_u32(&cm[tid]), b)) - sh) *
              ld_cluster_f32(mapa_shared(smem_u32(&cl[tid]), b));
    }
    __syncwarp();
    cluster_sync();  // every block has read the parts
    if (tid < 16) cm[tid] = mm, cl[tid] = ll;
  }
  __syncthreads();
  float sh[2], inv[2];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    sh[hh] = shift_of(cm[g + 8 * hh]);
    inv[hh] = 1.0f / cl[g + 8 * hh];
  }
  float* out = reinterpret_cast<float*>(a.out) + ((long long)blockIdx.z * a.Tq + s.q0 + row0) * a.ldo;
  const bool pairs = ((reinterpret_cast<uintptr_t>(a.out) & 7) | (a.ldo & 1)) == 0;  // rows of whole 8 bytes
  load_k(lo + warp * XW_KEYS, kf);
  for (int j0 = lo + warp * XW_KEYS; j0 < end; j0 += STEP) {
    const bool whole = pairs && j0 + XW_KEYS <= hi;
    {
      float c[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) scores8<KIND>(c[u], qf, kf[u][0], kf[u][1]);
      load_k(j0 + STEP, kf);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int row = g + 8 * hh;
        if (row0 + row >= s.lq) continue;
        float* dst = out + row * a.ldo + j0 + 2 * t;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float2 p;
          p.x = ex2_approx(fmaf(c[u][2 * hh], kScaleLog2, -sh[hh])) * inv[hh];
          p.y = ex2_approx(fmaf(c[u][2 * hh + 1], kScaleLog2, -sh[hh])) * inv[hh];
          if (whole) {
            *reinterpret_cast<float2*>(dst + 8 * u) = p;
          } else {
            const int j = j0 + 8 * u + 2 * t;
            if (j < end) dst[8 * u] = j < hi ? p.x : 0.f;
            if (j + 1 < end) dst[8 * u + 1] = j + 1 < hi ? p.y : 0.f;
          }
        }
      }
    }
  }
}

// Warps of a block and blocks of a cluster: enough warps in all to keep the
// loads of a full GPU in flight, about ten per SM (a warp has 8 KB on the way
// and waits about a microsecond for it), first by more warps in a block (joined
// in shared memory), then by more blocks, down to 8 keys a warp.  Measured, us,
// (warps x blocks) at 1500 keys unless stated: 12 tiles 4x1 11.5, 4x8 5.4,
// 16x8 5.5; 24 tiles 4x8 6.5, 16x4 6.0; 96 tiles 4x1 18.4, 4x4 12.4, 16x1 11.9,
// 16x4 19.3; 192 tiles 4x1 21.6, 8x1 17.6, 16x1 22.9; 384 tiles (5 rows) 4x1
// 30.2, 8x1 34.3, 4x2 36.5; 16 tiles at up to 30000 keys 4x8 41.0, 16x8 22.2; 4
// tiles at 30000 keys 16x8 19.3, 16x16 12.7.
template <int KIND, int NB>
static cudaError_t launch_rows(XattnArgs a, int n_seg, int max_k, int num_sms, cudaStream_t st) {
  // at least one tile: a longest segment of no rows is checked, too
  const int tiles = (int)std::max(((long long)a.max_q * a.G + 8 * NB - 1) / (8 * NB), 1LL), Hkv = a.H / a.G;
  const long long blocks = (long long)n_seg * tiles * Hkv, want = 10LL * num_sms;
  int W = 4;
  while (W < (NB == 1 ? 16 : 8) && blocks * W < want) W *= 2;
  a.splits = pick_splits(blocks * W, max_k, 8 * W, want, W == 4 ? 8 : 16);
  static WideClusters seen[2];
  a.splits = cap_splits(a.splits, [&] {
    if constexpr (NB == 1)
      if (W == 16) return holds_wide_cluster(xattn_rows_kernel<KIND, NB, 16>, 512, 0, seen[1]);
    return holds_wide_cluster(xattn_rows_kernel<KIND, NB, 8>, 256, 0, seen[0]);
  });
  const dim3 grid(n_seg * a.splits, tiles, Hkv);
  if (W == 4) return launch_cluster(xattn_rows_kernel<KIND, NB, 4>, grid, 128, 0, a.splits, st, a);
  if (W == 8) return launch_cluster(xattn_rows_kernel<KIND, NB, 8>, grid, 256, 0, a.splits, st, a);
  if constexpr (NB == 1) return launch_cluster(xattn_rows_kernel<KIND, NB, 16>, grid, 512, 0, a.splits, st, a);
  return cudaErrorInvalidValue;
}

// Up to 32 tokens the rows kernel, which reads the states once per 16 rows
// (tokens x shared heads); beyond, the tiles of 128 tokens of one query head.
// Both sides grow with the shared heads alike, so tokens alone decide.  On the
// device, rows / tiles, us, at 1500 states:
//   tokens                        16           32           48           64
//   1 segment,  G = 1  12 heads   10.5 / 13.7  10.1 / 13.8  14.7 / 13.9  11.4 / 13.9
//   8 segments, G = 1  12 heads   14.4 / 19.0  18.0 / 19.2  18.5 / 19.3  20.6 / 19.5
//   32,         G = 1  12 heads   28.1 / 42.9  43.4 / 43.4  61.2 / 44.3  79.3 / 45.0
//   32,         G = 5  20 heads   39.2 / 63.8  59.0 / 64.2  90.0 / 65.4  115 / 66.0
//   8 segments, G = 8  16 heads   14.7 / 19.2  19.0 / 19.2  23.0 / 19.4  33.8 / 19.5
//   32,         G = 8  16 heads   33.5 / 51.3  52.8 / 51.6  74.5 / 52.4  95.5 / 53.0
// The longest segment decides for the whole call: one prompt takes the calls
// of one token beside it along to the tiles.
cudaError_t launch_xattn(XattnArgs a, int n_seg, int max_k, bool f16, int num_sms, cudaStream_t st) {
  if (a.max_q > 32 && a.Tk > 0) return launch_xattn_tiles(a, n_seg, max_k, f16, num_sms, st);
  if ((long long)a.max_q * a.G <= 8)
    return f16 ? launch_rows<KIND_F16, 1>(a, n_seg, max_k, num_sms, st) : launch_rows<KIND_BF16, 1>(a, n_seg, max_k, num_sms, st);
  return f16 ? launch_rows<KIND_F16, 2>(a, n_seg, max_k, num_sms, st) : launch_rows<KIND_BF16, 2>(a, n_seg, max_k, num_sms, st);
}

// The same border for the weights (12 heads of 1500 states, rows / tiles, us, at
// 32, 48 and 64 tokens: 1 segment 6.4 / 12.1, 7.7 / 13.2, 7.9 / 12.3; 8 segments
// 16.4 / 28.6, 16.4 / 33.0, 30.8 / 28.8; 32 segments 56.9 / 63.6, 73.6 / 73.6,
// 90.8 / 69.3).  Without columns only the segments and heads are checked, which
// any kernel does.
cudaError_t launch_xattn_weights(XattnArgs a, int n_seg, int n_sel, bool f16, int num_sms, cudaStream_t st) {
  if (a.max_q > 32 && a.Tk > 0 && a.width > 0) return launch_xattn_weights_tiles(a, n_seg, n_sel, f16, num_sms, st);
  const int tiles = std::max((a.max_q + 15) / 16, 1);
  a.splits = pick_splits((long long)n_seg * tiles * n_sel, a.width, XW_WARPS * XW_KEYS, num_sms);
  const dim3 grid(n_seg * a.splits, tiles, n_sel);
  return f16 ? launch_cluster(xattn_weights_kernel<KIND_F16>, grid, 32 * XW_WARPS, 0, a.splits, st, a)
             : launch_cluster(xattn_weights_kernel<KIND_BF16>, grid, 32 * XW_WARPS, 0, a.splits, st, a);
}

}  // namespace asr
