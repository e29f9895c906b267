// Gradients of the norms around a residual stream (residual_norm_fwd.cu).  Bound by memory: dout, x_out,
// dx_out and y are read once, the gradients of the residual and of y written once.  The two row sums of
// each norm cost a barrier; the columns' sums (dgamma, dbeta, and two for the gate's and the post norm's
// gradients) stay in a thread's registers over its CTA's rows, leave as one partial row each, and are
// added in a fixed order by a second kernel.
#include "residual_norm.cuh"

namespace te {

namespace {

// ----------------------------------------------------------------------- backward --------

// Sums of two values over the CTA's G warps, added in warp order (the same bits in every thread); *bad
// becomes whether it was set in any thread.
template <int G>
__device__ __forceinline__ float2 row_sums(float a, float b, float2* red, bool* bad) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (G == 1) {
    *bad = __any_sync(0xffffffffu, *bad);
    return make_float2(a, b);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  *bad = __syncthreads_or(*bad) != 0;
  float2 t = red[0];
#pragma unroll
  for (int w = 1; w < G; ++w) {
    t.x += red[w].x;
    t.y += red[w].y;
  }
  return t;
}

// Warps of an SM, by their registers (four: LayerNorm on both sides, with four sums to a column).
__host__ __device__ constexpr int bwd_warps(int nv, bool four) { return nv >= 4 ? 8 : four && nv == 2 ? 12 : 16; }

// A CTA of G warps takes neighbouring rows.  With S1 = the sum of dx * phat and S2 = that of dx over the
// rows that share a gate (phat the normalized y, or y itself without a post norm), the gradients of the
// gate and of the post norm's gain and shift are
//   dgate = post_g * S1 + post_b * S2,  dpost_gamma = sum over gates of gate * S1,
//   dpost_beta = sum over gates of gate * S2,
// so a thread keeps two sums for these three.  They are written where a gate's rows end: the part of
// CTA c's rows that gate row g serves is slot c + g, which no other part has (c or g grows from one
// part to the next).
//
// A ring slot is [dout | x_out | dx_out | y]; where two slots would not fit, y is read from memory.
template <typename TY, typename TR, bool LN, bool POST, bool SUMS, int NV, int G>
__global__ void __launch_bounds__(G * 32, bwd_warps(NV, LN && POST) / G)
    residual_norm_bwd_kernel(ResidualNormBwdArgs a, int* status, int slots, bool y_in_ring) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int threads = G * 32;
  // (four sums, measured in bf16, us, with / without: 16384 x 8192 754 / 606, x 4096 250 / 282, x 1024 90 / 71; at 4096
  // bf16 spills 22 bytes with it, fp32, which was not compared, 260)
  constexpr bool KEEP = !(LN && POST) || (NV == 4 && G < 8);
  constexpr bool EARLY = KEEP && sizeof(TY) == 2;  // (fp32 vectors in waiting would spill)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[4][G];
  const int tid = threadIdx.x;
  const int units = int(a.H / 8);
  const float inv_h = 1.0f / float(a.H);
  const f32x2 shift2 = f2s(a.zero_centered_gamma ? 1.0f : 0.0f);
  const int64_t r0 = int64_t(blockIdx.x) * a.rows_per_cta;
  const int64_t r1 = r0 + a.rows_per_cta < a.M ? r0 + a.rows_per_cta : a.M;
  const uint32_t ty_bytes = uint32_t(a.H) * uint32_t(sizeof(TY)), tr_bytes = uint32_t(a.H) * uint32_t(sizeof(TR));
  const uint32_t at_x = ty_bytes, at_dxo = at_x + tr_bytes, at_y = at_dxo + (a.dx_out ? tr_bytes : 0);
  Ring ring(smem, at_y + (SUMS && y_in_ring ? ty_bytes : 0), slots);
  auto issue = [&](int64_t row, int slot) {
    const uint32_t bar = smem_u32(&ring.full[slot]);
    const uint32_t dst = smem_u32(ring.data) + uint32_t(slot) * ring.slot_bytes;
    mbar_expect_tx(bar, ring.slot_bytes);
    bulk_load(dst, static_cast<const TY*>(a.dout) + row * a.H, ty_bytes, bar);
    bulk_load(dst + at_x, static_cast<const TR*>(a.x_out) + row * a.H, tr_bytes, bar);
    if (a.dx_out) bulk_load(dst + at_dxo, static_cast<const TR*>(a.dx_out) + row * a.H, tr_bytes, bar);
    if (SUMS && y_in_ring) bulk_load(dst + at_y, static_cast<const TY*>(a.y) + row * a.H, ty_bytes, bar);
  };
  int64_t issued = r0;  // the next row to ask for (thread 0)
  if (tid == 0) {
    ring.init();
    for (int k = 0; k < slots && issued < r1; ++k) issue(issued++, k);
  }
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = tid + i * threads < units;
  __syncthreads();
  f32x2 ag[NV][4], ab[NV][4], s1[NV][4], s2[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int p = 0; p < 4; ++p) ag[i][p] = ab[i][p] = s1[i][p] = s2[i][p] = f2s(0.0f);
  int64_t gate_row = r0 / a.gate_rows;
  int64_t gate_end = (gate_row + 1) * a.gate_rows;
  // column sums [2][H] of this thread's units
  auto write = [&](float* dst, const f32x2 (&u)[NV][4], const f32x2 (&v)[NV][4], bool second) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (in[i]) {
        store8<float>(dst, (tid + i * threads) * 8, u[i]);
        if (second) store8<float>(dst + a.H, (tid + i * threads) * 8, v[i]);
      }
    }
  };
  int par = 0;
  bool bad = false;
  int64_t row = r0;
  // a row's statistics are asked for while the row before it is in work
  float n_mu = LN ? a.mu[row] : 0.0f, n_rs = a.rsigma[row];
  float n_pmu = POST && LN ? a.post_mu[row] : 0.0f, n_prs = POST ? a.post_rsigma[row] : 0.0f;
  for (; row < r1; ++row, par ^= 1) {
    const int64_t base = row * a.H + tid * 8;
    const float mu = n_mu, rs = n_rs, pmu = n_pmu, prs = n_prs;
    if (row + 1 < r1) {
      if (LN) n_mu = a.mu[row + 1];
      n_rs = a.rsigma[row + 1];
      if (POST && LN) n_pmu = a.post_mu[row + 1];
      if (POST) n_prs = a.post_rsigma[row + 1];
    }
    Param<TY> pa[NV], pb[NV];  // gamma, then the gate; the post norm's gain
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (EARLY && in[i]) pa[i].ask(a.gamma, (tid + i * threads) * 8);
    bad = !ring.wait(status);
    const uint8_t* here = ring.here();
    // xhat and dout * g, then phat and the gradient on its way, of each unit from one barrier to the next;
    // KEEP false, where they would spill beside four sums, takes what the slot still holds again instead
    f32x2 xh[KEEP ? NV : 1][4], dx[NV][4];
    f32x2 t1 = f2s(0.0f), t2 = f2s(0.0f);
    const f32x2 mu2 = f2s(mu), rs2 = f2s(rs), pmu2 = f2s(pmu), prs2 = f2s(prs);
    // dout, xhat and dout * g of unit i
    auto upstream = [&](int i, f32x2 (&d)[4], f32x2 (&h)[4], f32x2 (&dg)[4]) {
      const int u = (tid + i * threads) * 8;
      Unit<TY> dout;
      Unit<TR> x;
      dout.load(here, u);
      x.load(here + at_x, u);
      f32x2 g[4], xp[4];
      if (!EARLY) pa[i].ask(a.gamma, u);
      pa[i].get(g, 1.0f);
      dout.cvt(d);
      x.cvt(xp);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        h[p] = LN ? mul2(sub2(xp[p], mu2), rs2) : mul2(xp[p], rs2);
        dg[p] = mul2(d[p], add2(g[p], shift2));
      }
    };
    auto phat = [&](int i, f32x2 (&h)[4]) {
      Unit<TY> y;
      if (y_in_ring) y.load(here + at_y, (tid + i * threads) * 8);
      else y.load(a.y, base + i * threads * 8);
      y.cvt(h);
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (POST) h[p] = LN ? mul2(sub2(h[p], pmu2), prs2) : mul2(h[p], prs2);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (in[i]) {
        f32x2 d[4], dg[4], h[4];
        upstream(i, d, h, dg);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if (LN) t1 = add2(t1, dg[p]);
          t2 = fma2(dg[p], h[p], t2);
          ag[i][p] = fma2(d[p], h[p], ag[i][p]);
          if (LN) ab[i][p] = add2(ab[i][p], d[p]);
          if (KEEP) {
            xh[KEEP ? i : 0][p] = h[p];
            dx[i][p] = dg[p];
          }
        }
        if (SUMS && KEEP && EARLY) pa[i].ask(a.gate, gate_row * a.H + (tid + i * threads) * 8);
        if (POST && KEEP && EARLY) pb[i].ask(a.post_gamma, (tid + i * threads) * 8);
      }
    }
    const float2 m = row_sums<G>(f2lo(t1) + f2hi(t1), f2lo(t2) + f2hi(t2), red[par], &bad);
    if (bad) break;
    if (tid == 0 && row > r0 && issued < r1) {  // the slot of the row before
      fence_proxy_async_smem();
      issue(issued++, ring.before());
    }
    const f32x2 c1 = f2s(-rs * (m.x * inv_h)), c2 = f2s(-rs * (m.y * inv_h)), scale2 = f2s(a.residual_scale);
    t1 = t2 = f2s(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = (tid + i * threads) * 8;
      if (in[i]) {
        const int64_t at = base + i * threads * 8;
        f32x2 h[4];
        if (KEEP) {
#pragma unroll
          for (int p = 0; p < 4; ++p) h[p] = xh[KEEP ? i : 0][p];
        } else {
          f32x2 d[4];
          upstream(i, d, h, dx[i]);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p)
          dx[i][p] = fma2(h[p], c2, LN ? fma2(dx[i][p], rs2, c1) : mul2(dx[i][p], rs2));
        if (a.dx_out) {
          Unit<TR> dxo;
          f32x2 d[4];
          dxo.load(here + at_dxo, u);
          dxo.cvt(d);
#pragma unroll
          for (int p = 0; p < 4; ++p) dx[i][p] = add2(d[p], dx[i][p]);
        }
        if (a.dresidual) {
          f32x2 o[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) o[p] = mul2(dx[i][p], scale2);
          store8<TR>(a.dresidual, at, o);
        }
        if (SUMS) {
          phat(i, h);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            s1[i][p] = fma2(dx[i][p], h[p], s1[i][p]);
            if (POST && LN) s2[i][p] = add2(s2[i][p], dx[i][p]);
            if (KEEP) xh[KEEP ? i : 0][p] = h[p];
          }
          if (a.gate) {
            f32x2 gt[4];
            if (!KEEP || !EARLY) pa[i].ask(a.gate, gate_row * a.H + u);
            pa[i].get(gt, 1.0f);
#pragma unroll
            for (int p = 0; p < 4; ++p) dx[i][p] = mul2(dx[i][p], gt[p]);
          }
        }
        if (POST) {
          f32x2 g[4];
          if (!KEEP || !EARLY) pb[i].ask(a.post_gamma, u);
          pb[i].get(g, 1.0f);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            dx[i][p] = mul2(dx[i][p], add2(g[p], shift2));
            if (LN) t1 = add2(t1, dx[i][p]);
            t2 = fma2(dx[i][p], h[p], t2);
          }
        } else if (a.dy) {
          store8<TY>(a.dy, at, dx[i]);
        }
      }
    }
    if (POST) {
      const float2 n = row_sums<G>(f2lo(t1) + f2hi(t1), f2lo(t2) + f2hi(t2), red[2 + par], &bad);
      if (a.dy) {
        const f32x2 d1 = f2s(-prs * (n.x * inv_h)), d2 = f2s(-prs * (n.y * inv_h));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (in[i]) {
            f32x2 o[4], h[4];
            if (!KEEP) phat(i, h);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const f32x2 ph = KEEP ? xh[KEEP ? i : 0][p] : h[p];
              o[p] = fma2(ph, d2, LN ? fma2(dx[i][p], prs2, d1) : mul2(dx[i][p], prs2));
            }
            store8<TY>(a.dy, base + i * threads * 8, o);
          }
        }
      }
    }
    if (SUMS && (row + 1 == gate_end || row + 1 == r1)) {
      write(a.gate_partials + (int64_t(blockIdx.x) + gate_row) * 2 * a.H, s1, s2, POST && LN);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p) s1[i][p] = s2[i][p] = f2s(0.0f);
      ++gate_row;
      gate_end += a.gate_rows;
    }
    ring.next();
  }
  if (bad && tid == 0) ring.drain(row - r0, issued - r0, status);
  write(a.partials + int64_t(blockIdx.x) * 2 * a.H, ag, ab, LN);
}

// The columns' sums over the CTAs' partial rows, in a fixed order.  blockIdx.y: 0 dgamma and dbeta;
// 1 dpost_gamma and dpost_beta, from the parts of all gates, each by its gate; 2 and up the rows of
// dgate.  A CTA takes 64 columns, four to a lane of a half warp; its 32 half warps take the terms
// h, h + 32, ... and are added in order.
constexpr int kSumThreads = 512;
constexpr int kSumParts = kSumThreads / 16;
constexpr int kSumCols = 64;

struct Sum2 {
  float4 a, b;
};
__device__ __forceinline__ void add4(float4& t, const float4& v) {
  t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
}
__device__ __forceinline__ void fma4(float4& t, const float4& u, const float4& v) {
  t.x = fmaf(u.x, v.x, t.x); t.y = fmaf(u.y, v.y, t.y); t.z = fmaf(u.z, v.z, t.z); t.w = fmaf(u.w, v.w, t.w);
}

template <typename TY>
__device__ __forceinline__ float4 param4(const void* base, int64_t j, float shift, float fill) {
  if (base == nullptr) return make_float4(fill, fill, fill, fill);
  if (sizeof(TY) == 2) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + j));
    return make_float4(bf16_lo(w.x) + shift, bf16_hi(w.x) + shift, bf16_lo(w.y) + shift, bf16_hi(w.y) + shift);
  }
  const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + j));
  return make_float4(v.x + shift, v.y + shift, v.z + shift, v.w + shift);
}
__device__ __forceinline__ void put4(float* d, const float4& v) {
  d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
}

template <typename TY>
__global__ void __launch_bounds__(kSumThreads) residual_norm_bwd_sum_kernel(ResidualNormBwdArgs a, int ctas, bool ln) {
  __shared__ Sum2 box[kSumParts][16];
  // launched as a programmatic dependent of the kernel that writes the partials
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 15, h = threadIdx.x >> 4;
  const int64_t j = int64_t(blockIdx.x) * kSumCols + lane * 4;  // H is a multiple of 8
  const bool in = j < a.H;
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto at = [&](const float* p) { return *reinterpret_cast<const float4*>(p); };
  // the half warps' terms joined; the result is in half warp 0
  auto join = [&](Sum2 v) {
    __syncthreads();
    box[h][lane] = v;
    __syncthreads();
    if (h == 0) {
#pragma unroll 8
      for (int k = 1; k < kSumParts; ++k) {
        add4(v.a, box[k][lane].a);
        add4(v.b, box[k][lane].b);
      }
    }
    return v;
  };
  // the rows c0 + h, c0 + h + 32, ... up to c1 of [2][H] sums at p (many loads in flight: the terms are
  // few to a thread, and each comes from L2)
  auto rows = [&](const float* p, int c0, int c1, bool second) {
    Sum2 t{zero, zero};
    if (in) {
#pragma unroll 8
      for (int c = c0 + h; c <= c1; c += kSumParts) {
        const float* q = p + int64_t(c) * 2 * a.H + j;
        add4(t.a, at(q));
        if (second) add4(t.b, at(q + a.H));
      }
    }
    return t;
  };
  if (blockIdx.y == 0) {
    const Sum2 t = join(rows(a.partials, 0, ctas - 1, ln));
    if (h == 0 && in) {
      put4(a.dgamma + j, t.a);
      if (ln && a.dbeta) put4(a.dbeta + j, t.b);
    }
    return;
  }
  const bool post = a.post_gamma != nullptr, two = post && ln;
  const int gate_rows = int(a.gate_rows), per_cta = int(a.rows_per_cta), m = int(a.M), gates = m / gate_rows;
  if (blockIdx.y == 1) {
    if (!a.dpost_gamma && !(two && a.dpost_beta)) return;
    Sum2 t{zero, zero};
    if (gates <= kSumParts) {  // gate by gate: its parts are neighbours
      for (int g = 0; g < gates; ++g) {
        const Sum2 u = rows(a.gate_partials + int64_t(g) * 2 * a.H, int(int64_t(g) * gate_rows / per_cta),
                            int((int64_t(g + 1) * gate_rows - 1) / per_cta), two);
        const float4 gt = in ? param4<TY>(a.gate, int64_t(g) * a.H + j, 0.0f, 1.0f) : zero;
        fma4(t.a, gt, u.a);
        fma4(t.b, gt, u.b);
      }
    } else {  // CTA by CTA, which hold one gate's rows or several
      if (in) {
        for (int c = h; c < ctas; c += kSumParts) {
          const int last = min((c + 1) * per_cta, m) - 1;
          for (int g = c * per_cta / gate_rows; g <= last / gate_rows; ++g) {
            const float4 gt = param4<TY>(a.gate, int64_t(g) * a.H + j, 0.0f, 1.0f);
            const float* p = a.gate_partials + int64_t(c + g) * 2 * a.H + j;
            fma4(t.a, gt, at(p));
            if (two) fma4(t.b, gt, at(p + a.H));
          }
        }
      }
    }
    t = join(t);
    if (h == 0 && in) {
      if (a.dpost_gamma) put4(a.dpost_gamma + j, t.a);
      if (two && a.dpost_beta) put4(a.dpost_beta + j, t.b);
    }
    return;
  }
  const float shift = a.zero_centered_gamma ? 1.0f : 0.0f;
  const float4 g1 = in && post ? param4<TY>(a.post_gamma, j, shift, 1.0f) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  const float4 b1 = in && two ? param4<TY>(a.post_beta, j, 0.0f, 0.0f) : zero;
  for (int g = int(blockIdx.y) - 2; g < gates; g += int(gridDim.y) - 2) {
    const int c0 = int(int64_t(g) * gate_rows / per_cta), c1 = int((int64_t(g + 1) * gate_rows - 1) / per_cta);
    const Sum2 t = join(rows(a.gate_partials + int64_t(g) * 2 * a.H, c0, c1, two));
    if (h == 0 && in) {
      float4 o = zero;
      fma4(o, g1, t.a);
      if (two) fma4(o, b1, t.b);
      put4(a.dgate + int64_t(g) * a.H + j, o);
    }
  }
}

// Warps to a row and units to a thread, by the row's units.
struct BwdShape {
  int nv, warps;
  int64_t ctas, rows_per_cta;
};
BwdShape bwd_shape(int64_t M, int64_t H, bool four) {
  const int64_t units = H / 8;
  BwdShape s;
  s.nv = units <= 32 ? 1 : units <= 128 ? 2 : 4;
  s.warps = units <= 64 ? 1 : units <= 256 ? 2 : units <= 512 ? 4 : 8;
  const int64_t n = int64_t(num_sms()) * (bwd_warps(s.nv, four) / s.warps);
  s.rows_per_cta = M > n ? ceil_div(M, n) : 1;
  s.ctas = ceil_div(M, s.rows_per_cta);
  return s;
}

template <typename TY, typename TR, bool LN, bool POST, bool SUMS, int NV, int G>
te_status bwd_kernel(const ResidualNormBwdArgs& a, const BwdShape& sh, cudaStream_t s) {
  static PerDevice<bool> attr_done;
  auto kernel = residual_norm_bwd_kernel<TY, TR, LN, POST, SUMS, NV, G>;
  if (!allow_smem(kernel, attr_done)) return TE_ERR_CUDA;
  const size_t y = SUMS ? size_t(a.H) * sizeof(TY) : 0;
  const size_t rest = size_t(a.H) * (sizeof(TY) + (a.dx_out ? 2 : 1) * sizeof(TR));
  // (three slots for rows of 4 warps and more: 139 us for 147, LayerNorm with a gate at 16384 x 4096; for
  // shorter ones two: 80 for 87 at 2048)
  const int most = G >= 4 ? 3 : 2;
  RingShape ring = ring_shape(bwd_warps(NV, LN && POST) / G, rest + y, most);
  const bool y_in_ring = ring.ctas != 0;
  if (!y_in_ring) ring = ring_shape(1, rest, most);
  if (ring.ctas == 0) return TE_ERR_UNSUPPORTED;
  const size_t bytes = kHeader + size_t(ring.slots) * (rest + (y_in_ring ? y : 0));
  kernel<<<unsigned(sh.ctas), G * 32, bytes, s>>>(a, device_status_ptr(), ring.slots, y_in_ring);
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

template <typename TY, typename TR, bool LN, bool POST, bool SUMS>
te_status bwd_launch(ResidualNormBwdArgs a, cudaStream_t s) {
  const BwdShape sh = bwd_shape(a.M, a.H, LN && POST);
  a.rows_per_cta = sh.rows_per_cta;
  a.gate_partials = a.partials + sh.ctas * 2 * a.H;
  te_status st;
  if (sh.nv == 1) st = bwd_kernel<TY, TR, LN, POST, SUMS, 1, 1>(a, sh, s);
  else if (sh.nv == 2 && sh.warps == 1) st = bwd_kernel<TY, TR, LN, POST, SUMS, 2, 1>(a, sh, s);
  else if (sh.nv == 2) st = bwd_kernel<TY, TR, LN, POST, SUMS, 2, 2>(a, sh, s);
  else if (sh.warps == 2) st = bwd_kernel<TY, TR, LN, POST, SUMS, 4, 2>(a, sh, s);
  else if (sh.warps == 4) st = bwd_kernel<TY, TR, LN, POST, SUMS, 4, 4>(a, sh, s);
  else st = bwd_kernel<TY, TR, LN, POST, SUMS, 4, 8>(a, sh, s);
  if (st != TE_OK) return st;
  const int64_t gates = a.M / a.gate_rows;
  const unsigned rows = !SUMS ? 1 : a.dgate ? unsigned(2 + (gates < 4096 ? gates : 4096)) : 2;
  return launch_dependent(residual_norm_bwd_sum_kernel<TY>, dim3(unsigned(ceil_div(a.H, kSumCols)), rows),
                          dim3(kSumThreads), s, a, int(sh.ctas), LN);
}

template <typename TY, typename TR, bool LN>
te_status bwd_norm(const ResidualNormBwdArgs& a, cudaStream_t s) {
  if (a.post_gamma) return bwd_launch<TY, TR, LN, true, true>(a, s);
  return a.gate ? bwd_launch<TY, TR, LN, false, true>(a, s) : bwd_launch<TY, TR, LN, false, false>(a, s);
}

template <typename TY, typename TR>
te_status bwd_types(const ResidualNormBwdArgs& a, cudaStream_t s) {
  return a.norm_type == TE_LAYERNORM ? bwd_norm<TY, TR, true>(a, s) : bwd_norm<TY, TR, false>(a, s);
}

}  // namespace

size_t residual_norm_bwd_workspace(int64_t M, int64_t H, int64_t gates) {
  if (M <= 0 || H <= 0) return 0;
  const int64_t ctas = bwd_shape(M, H, false).ctas;  // (no fewer than with four sums)
  return size_t(2 * ctas + (gates > 0 ? gates : 1)) * 2 * size_t(H) * sizeof(float);
}

te_status launch_residual_norm_bwd(const ResidualNormBwdArgs& a, cudaStream_t s) {
  if (a.M == 0) return TE_OK;
  ProfileScope prof(TE_KERNEL_NORM_BWD, s);
  if (a.dtype == TE_F32) return bwd_types<float, float>(a, s);
  return a.residual_dtype == TE_F32 ? bwd_types<__nv_bfloat16, float>(a, s)
                                    : bwd_types<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace te
