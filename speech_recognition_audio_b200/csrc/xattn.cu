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
// Few rows: a tile of 16 rows (tokens x shared heads) per block, where the
// time is that of reading the states once.  The keys are split over the
// warps of a block and the blocks of a cluster, each warp keeping a running
// maximum and sum of its own; the parts are joined in a fixed order through
// shared and distributed shared memory.  Keys and values go from global
// memory straight into mma.sync operand registers (no shared memory on the
// way): a contraction may visit its terms in any order, so lane (g, t) of the
// fragment layout takes whole 16-byte pieces of a key row and the query
// fragments follow the same order, and the values' columns are permuted the
// same way.  mma.sync rather than tcgen05: a 128-row tile would be all but
// empty, and the tensor pipe is idle most of the time either way.
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
// Query fragments of 16 rows (row r of the tile: token r / G, head kvh G + r % G):
// lane (g, t) holds, of rows g and g + 8, elements 8 t .. 8 t + 7 and
// 32 + 8 t .. 32 + 8 t + 7, i.e. k step s is elements 32 (s / 2) + 8 t + 4 (s % 2) + 0..3.
__device__ __forceinline__ void load_q16(const XattnArgs& a, const Segment& s, int row0, int kvh, int G, int lane,
                                         uint32_t (*qf)[4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int r = row0 + g + 8 * hh, tok = r / G, h = kvh * G + (r - tok * G);
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

constexpr int XS_WARPS = 4, XS_KEYS = 32;  // warps of a block, keys of a warp's step

}  // namespace

template <int KIND>
__global__ void __launch_bounds__(32 * XS_WARPS, 3) xattn_rows_kernel(const XattnArgs a) {
  __shared__ __align__(16) float so[XS_WARPS][16][68];  // rows padded against bank conflicts
  __shared__ float sm[XS_WARPS][16], sl[XS_WARPS][16];
  __shared__ float cm[16], cl[16];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int S = a.splits, seg = blockIdx.x / S, rank = blockIdx.x - seg * S;
  const int row0 = blockIdx.y * 16, kvh = blockIdx.z, G = a.G;
  const Segment s = load_segment(a, seg, tid == 0);
  if (!s.ok || row0 >= s.lq * G) return;  // the same for every block of the cluster

  uint32_t qf[4][4];
  load_q16(a, s, row0, kvh, G, lane, qf);
  // this block's keys, in whole steps of a warp
  const int steps = (s.lk + XS_KEYS - 1) / XS_KEYS;
  const int lo = rank * steps / S * XS_KEYS, hi = min((rank + 1) * steps / S * XS_KEYS, s.lk);
  const uint16_t* kp = reinterpret_cast<const uint16_t*>(a.k) + (long long)s.k0 * a.ldk + 64 * kvh + 8 * t;
  const uint16_t* vp = reinterpret_cast<const uint16_t*>(a.v) + (long long)s.k0 * a.ldv + 64 * kvh + 8 * g;
  float o[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  for (int j0 = lo + warp * XS_KEYS; j0 < hi; j0 += XS_WARPS * XS_KEYS) {
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
    float c[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) scores8<KIND>(c[u], qf, kf[u][0], kf[u][1]);
    // keys past the end never count, whatever the arrays hold there
    if (j0 + XS_KEYS > hi) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + 8 * u + 2 * t + (i & 1) >= hi) c[u][i] = -INFINITY;
    }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < 4; ++u) mx = fmaxf(mx, fmaxf(c[u][2 * hh], c[u][2 * hh + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      mx = fmaxf(m[hh], mx * kScaleLog2);
      const float sh = shift_of(mx), corr = ex2_approx(m[hh] - sh);
      m[hh] = mx;
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 2 * hh; i < 2 * hh + 2; ++i) {
          c[u][i] = ex2_approx(fmaf(c[u][i], kScaleLog2, -sh));
          sum += c[u][i];
        }
      l[hh] = l[hh] * corr + sum;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j][2 * hh] *= corr, o[j][2 * hh + 1] *= corr;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // probabilities rounded to the values' type, the operand type of the product
      const uint32_t pf[4] = {pack2_16<KIND>(c[2 * u][0], c[2 * u][1]), pack2_16<KIND>(c[2 * u][2], c[2 * u][3]),
                              pack2_16<KIND>(c[2 * u + 1][0], c[2 * u + 1][1]),
                              pack2_16<KIND>(c[2 * u + 1][2], c[2 * u + 1][3])};
      const uint32_t* v0 = reinterpret_cast<const uint32_t*>(&vf[u][0]);
      const uint32_t* v1 = reinterpret_cast<const uint32_t*>(&vf[u][1]);
      const uint32_t* v2 = reinterpret_cast<const uint32_t*>(&vf[u][2]);
      const uint32_t* v3 = reinterpret_cast<const uint32_t*>(&vf[u][3]);
      // column n of product j is element 8 n + j
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        mma16<KIND>(o[j], pf, __byte_perm(v0[j >> 1], v1[j >> 1], sel), __byte_perm(v2[j >> 1], v3[j >> 1], sel));
      }
    }
  }
  // this warp's part: lane (g, t) holds elements 16 t + j and 16 t + 8 + j of rows g, g + 8
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
    l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
    if (t == 0) sm[warp][g + 8 * hh] = m[hh], sl[warp][g + 8 * hh] = l[hh];
    float* dst = &so[warp][g + 8 * hh][16 * t];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<float4*>(dst + j) = make_float4(o[j][2 * hh], o[j + 1][2 * hh], o[j + 2][2 * hh], o[j + 3][2 * hh]);
      *reinterpret_cast<float4*>(dst + 8 + j) =
          make_float4(o[j][2 * hh + 1], o[j + 1][2 * hh + 1], o[j + 2][2 * hh + 1], o[j + 3][2 * hh + 1]);
    }
  }
  __syncthreads();
  // join the warps: thread (row, 8 elements); the result replaces warp 0's part
  const int row = tid >> 3, c8 = 8 * (tid & 7);
  float acc[8];
  {
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < XS_WARPS; ++w) mm = fmaxf(mm, sm[w][row]);
    const float sh = shift_of(mm);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < XS_WARPS; ++w) {
      const float f = ex2_approx(sm[w][row] - sh);
      ll += f * sl[w][row];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(f, so[w][row][c8 + i], acc[i]);
    }
    if (S > 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) so[0][row][c8 + i] = acc[i];  // only this thread reads or writes these
      if ((tid & 7) == 0) cm[row] = mm, cl[row] = ll;
      __syncwarp();
      cluster_sync();
      // join the blocks: each takes a share of the (row, 8 elements) pieces
      const int mine = tid * S + rank;
      if (mine < 128) {
        const int r = mine >> 3, e = 8 * (mine & 7);
        const uint32_t am = smem_u32(&cm[r]), al = smem_u32(&cl[r]), ao = smem_u32(&so[0][r][e]);
        mm = -INFINITY;
        ll = 0.f;
        for (int b = 0; b < S; ++b) mm = fmaxf(mm, ld_cluster_f32(mapa_shared(am, b)));
        const float sh2 = shift_of(mm);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        for (int b = 0; b < S; ++b) {
          const float f = ex2_approx(ld_cluster_f32(mapa_shared(am, b)) - sh2);
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
      if (mine >= 128) return;
    }
    const int mine = S > 1 ? tid * S + rank : tid;
    const int rr = row0 + (mine >> 3), e = 8 * (mine & 7);
    const int tok = rr / G, h = kvh * G + (rr - tok * G);
    if (tok < s.lq) {
      const float inv = s.lk > 0 ? 1.0f / ll : 0.f;  // no states: zeros
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] *= inv;
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + (long long)(s.q0 + tok) * a.ldo + 64 * h + e) =
          pack8_16<KIND>(acc);
    }
  }
}

// Attention weights of one selected head over RT tiles of 16 rows per block.
// Two passes over the keys (the second finds them in L2): running maximum and
// sum, joined over warps and the blocks of the cluster; then the scores again,
// written as probabilities in 32 bits.  A row's 8 keys of a step are one
// 32-byte sector of the output.
constexpr int XW_WARPS = 8, XW_KEYS = 32;

template <int KIND, int RT>
__global__ void __launch_bounds__(32 * XW_WARPS, 2) xattn_weights_kernel(const XattnArgs a) {
  __shared__ float sm[XW_WARPS][16 * RT], sl[XW_WARPS][16 * RT];
  __shared__ float cm[16 * RT], cl[16 * RT];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int S = a.splits, seg = blockIdx.x / S, rank = blockIdx.x - seg * S;
  const int row0 = blockIdx.y * 16 * RT;
  const Segment s = load_segment(a, seg, tid == 0);
  const int h = a.heads ? __ldg(a.heads + blockIdx.z) : blockIdx.z;
  const bool head_ok = h >= 0 && h < a.H;
  if (!head_ok && tid == 0) atomicCAS(a.status, 0, DEV_BAD_SEGMENT);
  if (!s.ok || !head_ok || row0 >= s.lq) return;  // the same for every block of the cluster

  uint32_t qf[RT][4][4];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    // rows are tokens of head h: a tile of "G = 1" rows of a head array that starts at h
    load_q16(a, s, row0 + 16 * r, h, 1, lane, qf[r]);
  }
  const uint16_t* kp = reinterpret_cast<const uint16_t*>(a.k) + (long long)s.k0 * a.ldk + 64 * (h / a.G) + 8 * t;
  const int steps = (a.width + XW_KEYS - 1) / XW_KEYS;
  const int lo = rank * steps / S * XW_KEYS, end = min((rank + 1) * steps / S * XW_KEYS, a.width);
  const int hi = min(end, s.lk);

  float m[RT][2], l[RT][2];
#pragma unroll
  for (int r = 0; r < RT; ++r) m[r][0] = m[r][1] = -INFINITY, l[r][0] = l[r][1] = 0.f;
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
    if (RT == 1) load_k(j0 + STEP, kn);  // registers for the next step's keys only beside few rows
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float c[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) scores8<KIND>(c[u], qf[r], kf[u][0], kf[u][1]);
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
        const float mn = fmaxf(m[r][hh], mx * kScaleLog2), sh = shift_of(mn);
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 2 * hh; i < 2 * hh + 2; ++i) sum += ex2_approx(fmaf(c[u][i], kScaleLog2, -sh));
        l[r][hh] = l[r][hh] * ex2_approx(m[r][hh] - sh) + sum;
        m[r][hh] = mn;
      }
    }
    if (RT == 1) {
#pragma unroll
      for (int u = 0; u < 4; ++u) kf[u][0] = kn[u][0], kf[u][1] = kn[u][1];
    } else {
      load_k(j0 + STEP, kf);
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float mm = m[r][hh];
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 2));
      float ll = l[r][hh] * ex2_approx(m[r][hh] - shift_of(mm));
      ll += __shfl_xor_sync(0xffffffffu, ll, 1);
      ll += __shfl_xor_sync(0xffffffffu, ll, 2);
      if (t == 0) sm[warp][16 * r + g + 8 * hh] = mm, sl[warp][16 * r + g + 8 * hh] = ll;
    }
  __syncthreads();
  if (tid < 16 * RT) {
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
    if (tid < 16 * RT) {
      for (int b = 0; b < S; ++b) mm = fmaxf(mm, ld_cluster_f32(mapa_shared(smem_u32(&cm[tid]), b)));
      const float sh = shift_of(mm);
      for (int b = 0; b < S; ++b)
        ll += ex2_approx(ld_cluster_f32(mapa_shared(smem_u32(&cm[tid]), b)) - sh) *
              ld_cluster_f32(mapa_shared(smem_u32(&cl[tid]), b));
    }
    __syncwarp();
    cluster_sync();  // every block has read the parts
    if (tid < 16 * RT) cm[tid] = mm, cl[tid] = ll;
  }
  __syncthreads();
  float sh[RT][2], inv[RT][2];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      sh[r][hh] = shift_of(cm[16 * r + g + 8 * hh]);
      inv[r][hh] = 1.0f / cl[16 * r + g + 8 * hh];
    }
  float* out = reinterpret_cast<float*>(a.out) + ((long long)blockIdx.z * a.Tq + s.q0 + row0) * a.ldo;
  const bool pairs = ((reinterpret_cast<uintptr_t>(a.out) & 7) | (a.ldo & 1)) == 0;  // rows of whole 8 bytes
  load_k(lo + warp * XW_KEYS, kf);
  for (int j0 = lo + warp * XW_KEYS; j0 < end; j0 += STEP) {
    const bool whole = pairs && j0 + XW_KEYS <= hi;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float c[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) scores8<KIND>(c[u], qf[r], kf[u][0], kf[u][1]);
      if (RT == 1 || r == RT - 1) load_k(j0 + STEP, kf);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int row = 16 * r + g + 8 * hh;
        if (row0 + row >= s.lq) continue;
        float* dst = out + row * a.ldo + j0 + 2 * t;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float2 p;
          p.x = ex2_approx(fmaf(c[u][2 * hh], kScaleLog2, -sh[r][hh])) * inv[r][hh];
          p.y = ex2_approx(fmaf(c[u][2 * hh + 1], kScaleLog2, -sh[r][hh])) * inv[r][hh];
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

cudaError_t launch_xattn(XattnArgs a, int n_seg, int max_k, bool f16, int num_sms, cudaStream_t st) {
  if (a.max_q > 32 && a.Tk > 0) return launch_xattn_tiles(a, n_seg, max_k, f16, num_sms, st);
  const int tiles = (int)(((long long)a.max_q * a.G + 15) / 16), Hkv = a.H / a.G;
  a.splits = pick_splits((long long)n_seg * tiles * Hkv, max_k, XS_WARPS * XS_KEYS, 2LL * num_sms);
  const dim3 grid(n_seg * a.splits, tiles, Hkv);
  return f16 ? launch_cluster(xattn_rows_kernel<KIND_F16>, grid, 32 * XS_WARPS, 0, a.splits, st, a)
             : launch_cluster(xattn_rows_kernel<KIND_BF16>, grid, 32 * XS_WARPS, 0, a.splits, st, a);
}

cudaError_t launch_xattn_weights(XattnArgs a, int n_seg, int n_sel, bool f16, int num_sms, cudaStream_t st) {
  if (a.max_q > 32 && a.Tk > 0) return launch_xattn_weights_tiles(a, n_seg, n_sel, f16, st);
  const bool wide = a.max_q > 16;
  const int rows = wide ? 64 : 16, tiles = (a.max_q + rows - 1) / rows;
  a.splits = pick_splits((long long)n_seg * tiles * n_sel, a.width, XW_WARPS * XW_KEYS, num_sms);
  const dim3 grid(n_seg * a.splits, tiles, n_sel);
  if (wide)
    return f16 ? launch_cluster(xattn_weights_kernel<KIND_F16, 4>, grid, 32 * XW_WARPS, 0, a.splits, st, a)
               : launch_cluster(xattn_weights_kernel<KIND_BF16, 4>, grid, 32 * XW_WARPS, 0, a.splits, st, a);
  return f16 ? launch_cluster(xattn_weights_kernel<KIND_F16, 1>, grid, 32 * XW_WARPS, 0, a.splits, st, a)
             : launch_cluster(xattn_weights_kernel<KIND_BF16, 1>, grid, 32 * XW_WARPS, 0, a.splits, st, a);
}

}  // namespace asr
