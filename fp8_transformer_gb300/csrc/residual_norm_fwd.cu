// The norms around a residual stream (an addition of this library; the norm itself is that of the
// TransformerEngine JAX "LayerNorm MLP" page, Description, forward step (1)):
//   p = norm(y; post_gamma, post_beta) or y,  x_out = a * residual + gate * p,  out = norm(x_out)
// Unfused this is four passes over rows in memory; here a row is read once, stays in registers, and its
// two results are written once, which bounds it.
//
// A row belongs to a CTA of 1 to 8 warps, each thread holding up to 4 units of 8 neighbouring elements:
// the fewer threads to a row, the fewer instructions its sums cost (rows on twice the threads, half the
// units each: 131 for 95 us, LayerNorm at 16384 x 4096).  Rows arrive by bulk copies in a ring of
// shared-memory slots, a slot for one row of each input, as far ahead as the ring allows.
#include "residual_norm.cuh"

namespace te {

namespace {

// ----------------------------------------------------------------------- forward ---------

constexpr int kMaxWarps = 32;

// (mean, 1 / sqrt(variance + eps)) of a row held by the CTA's G warps (G = 0: as many as it has), whose
// warp w holds count[w] elements.  LayerNorm: each warp takes its own mean, then the squares about it,
// and the warps' (count, mean, squares) are joined about the row's mean, so that no sum of squares of a
// large mean is ever formed and one barrier serves both.
template <bool LN, int NV, int G>
__device__ __forceinline__ float2 row_stats(const f32x2 (&v)[NV][4], const bool (&in)[NV], float inv_h, float eps,
                                            float2* red, const float* count, bool* bad) {
  const int lane = threadIdx.x & 31, warp = G == 1 ? 0 : threadIdx.x >> 5, warps = G ? G : blockDim.x >> 5;
  float mean_w = 0.0f;
  if (LN) {
    f32x2 s = f2s(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) s = add2(s, sum8(v[i]));  // (units outside the row are zero)
    mean_w = warp_sum(f2lo(s) + f2hi(s)) * count[kMaxWarps + warp];
  }
  const f32x2 m2 = f2s(mean_w);
  f32x2 q0 = f2s(0.0f), q1 = f2s(0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!LN || in[i]) {
#pragma unroll
      for (int p = 0; p < 4; p += 2) {
        const f32x2 d0 = LN ? sub2(v[i][p], m2) : v[i][p], d1 = LN ? sub2(v[i][p + 1], m2) : v[i][p + 1];
        q0 = fma2(d0, d0, q0);
        q1 = fma2(d1, d1, q1);
      }
    }
  }
  q0 = add2(q0, q1);
  const float sq = warp_sum(f2lo(q0) + f2hi(q0));
  if (G == 1) {
    *bad = __any_sync(0xffffffffu, *bad);
    return make_float2(mean_w, rsqrtf(sq * inv_h + eps));
  }
  if (lane == 0) red[warp] = make_float2(mean_w, sq);
  *bad = __syncthreads_or(*bad) != 0;
  float mean = 0.0f, var = 0.0f;
  if (LN) {
#pragma unroll
    for (int w = 0; w < warps; ++w) mean = fmaf(count[w], red[w].x, mean);
    mean *= inv_h;
  }
#pragma unroll
  for (int w = 0; w < warps; ++w) {
    const float2 r = red[w];
    const float d = r.x - mean;
    var += LN ? fmaf(count[w], d * d, r.y) : r.y;
  }
  return make_float2(mean, rsqrtf(fmaf(var, inv_h, eps)));
}

// A unit normalized with the row's (mean, 1 / deviation), its gain (plus shift) and beta.
template <bool LN, typename T>
__device__ __forceinline__ void normalize(f32x2 (&x)[4], float2 st, const Param<T>& gain, const Param<T>& beta,
                                          float shift) {
  f32x2 g[4], b[4];
  gain.get(g, 1.0f);
  if (LN) beta.get(b, 0.0f);
  const f32x2 mean2 = f2s(st.x), rs2 = f2s(st.y), srs2 = f2s(shift * st.y);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const f32x2 k = fma2(g[p], rs2, srs2);  // (g + shift) / deviation
    x[p] = LN ? fma2(sub2(x[p], mean2), k, b[p]) : mul2(x[p], k);
  }
}

__host__ __device__ constexpr int fwd_threads(int g) { return g == 0 ? 1024 : g * 32; }
__host__ __device__ constexpr int fwd_ctas(int g) { return g == 0 ? 1 : 16 / g; }  // on an SM

// G warps to a row (one CTA), NV units to a thread, rows through the ring.  G = 0: a few long rows, as
// many warps to each as its units (NV = 1) ask for, and loads straight into registers.
template <typename TY, typename TR, bool LN, bool POST, int NV, int G>
__global__ void __launch_bounds__(fwd_threads(G), fwd_ctas(G))
    residual_norm_fwd_kernel(ResidualNormArgs a, int* status, int slots) {
  // the kernel after this one may launch its setup now (it waits for this grid's completion)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr bool RING = G != 0;
  constexpr bool EARLY = sizeof(TY) == 2;  // (fp32 vectors in waiting would spill)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[4][G == 1 ? 1 : kMaxWarps];
  __shared__ float count[2 * kMaxWarps];  // elements that each warp holds, and one over them
  const int tid = threadIdx.x, threads = G ? G * 32 : blockDim.x;
  const int units = int(a.H / 8);
  const uint32_t y_bytes = uint32_t(a.H) * uint32_t(sizeof(TY)), r_bytes = uint32_t(a.H) * uint32_t(sizeof(TR));
  Ring ring(smem, y_bytes + r_bytes, slots);
  const int64_t step = gridDim.x;
  auto issue = [&](int64_t row, int slot) {
    const uint32_t bar = smem_u32(&ring.full[slot]);
    const uint32_t dst = smem_u32(ring.data) + uint32_t(slot) * ring.slot_bytes;
    mbar_expect_tx(bar, ring.slot_bytes);
    bulk_load(dst, static_cast<const TY*>(a.y) + row * a.H, y_bytes, bar);
    bulk_load(dst + y_bytes, static_cast<const TR*>(a.residual) + row * a.H, r_bytes, bar);
  };
  int64_t issued = blockIdx.x;  // the next row to ask for (thread 0)
  if (RING && tid == 0) {
    ring.init();
    for (int k = 0; k < slots && issued < a.M; ++k, issued += step) issue(issued, k);
  }
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = tid + i * threads < units;
  if (tid < kMaxWarps) {
    int n = 0;
    for (int i = 0; i < NV; ++i) n += max(0, min(32, units - (tid * 32 + i * threads)));
    count[tid] = float(8 * n);
    count[kMaxWarps + tid] = n > 0 ? 1.0f / float(8 * n) : 0.0f;
  }
  __syncthreads();
  const CastState cs = cast_begin(a.cast);
  const int kind = out_kind(cs);
  const bool want_amax = a.cast.amax_out != nullptr;
  const float inv_h = 1.0f / float(a.H);
  const float shift = a.zero_centered_gamma ? 1.0f : 0.0f;
  const f32x2 scale2 = f2s(a.residual_scale);
  float amax = 0.0f;
  int par = 0;
  bool bad = false;
  int64_t row = blockIdx.x;
  for (; row < a.M; row += step, par ^= 1) {
    const int64_t base = row * a.H + tid * 8;
    const int64_t gate_at = a.gate ? row / a.gate_rows * a.H : 0;
    Unit<TY> y[NV];
    Unit<TR> r[NV];  // (ring: read from the slot when it is needed)
    Param<TY> gate[NV], g[NV], b[NV];
    if (RING) bad = !ring.wait(status);
    const uint8_t* here = ring.here();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = (tid + i * threads) * 8;
      y[i].zero();
      if (in[i]) {
        if (RING) {
          y[i].load(here, u);
        } else {
          y[i].load(a.y, base + i * threads * 8);
          r[i].load(a.residual, base + i * threads * 8);
        }
        if (EARLY) gate[i].ask(a.gate, gate_at + u);
        if (POST && EARLY) {
          g[i].ask(a.post_gamma, u);
          if (LN) b[i].ask(a.post_beta, u);
        }
      }
    }
    f32x2 x[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) y[i].cvt(x[i]);
    if (POST) {
      const float2 st = row_stats<LN, NV, G>(x, in, inv_h, a.eps, red[2 + par], count, &bad);
      if (tid == 0) {
        if (a.post_mu) a.post_mu[row] = st.x;
        if (a.post_rsigma) a.post_rsigma[row] = st.y;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (in[i]) {
          if (!EARLY) {
            g[i].ask(a.post_gamma, (tid + i * threads) * 8);
            if (LN) b[i].ask(a.post_beta, (tid + i * threads) * 8);
          }
          normalize<LN>(x[i], st, g[i], b[i], shift);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (in[i]) {
        const int u = (tid + i * threads) * 8;
        f32x2 rp[4];
        if (RING) r[i].load(here + y_bytes, u);
        r[i].cvt(rp);
        if (a.gate) {
          f32x2 q[4];
          if (!EARLY) gate[i].ask(a.gate, gate_at + u);
          gate[i].get(q, 1.0f);
#pragma unroll
          for (int p = 0; p < 4; ++p) x[i][p] = mul2(x[i][p], q[p]);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) x[i][p] = fma2(scale2, rp[p], x[i][p]);
        if (kind != OUT_NONE && !bad) store8<TR>(a.x_out, base + i * threads * 8, x[i]);
        if (EARLY) {
          g[i].ask(a.gamma, u);
          if (LN) b[i].ask(a.beta, u);
        }
      }
    }
    const float2 st = row_stats<LN, NV, G>(x, in, inv_h, a.eps, red[par], count, &bad);
    if (bad) break;
    if (RING && tid == 0 && issued < a.M) {  // every thread has what it reads of this row
      fence_proxy_async_smem();
      issue(issued, ring.slot);
      issued += step;
    }
    if (tid == 0) {
      if (a.mu) a.mu[row] = st.x;
      if (a.rsigma) a.rsigma[row] = st.y;
    }
    auto finish = [&](auto tag) {
      constexpr int OUT = decltype(tag)::value;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (in[i]) {
          if (!EARLY) {
            g[i].ask(a.gamma, (tid + i * threads) * 8);
            if (LN) b[i].ask(a.beta, (tid + i * threads) * 8);
          }
          normalize<LN>(x[i], st, g[i], b[i], shift);
          if (want_amax) {
#pragma unroll
            for (int p = 0; p < 4; ++p) amax = absmax2(amax, x[i][p]);
          }
          const float o[8] = {x[i][0].x, x[i][0].y, x[i][1].x, x[i][1].y, x[i][2].x, x[i][2].y, x[i][3].x, x[i][3].y};
          store_out<OUT, 8>(a.out, base + i * threads * 8, o, cs);
        }
      }
    };
    switch (kind) {
      case OUT_F32: finish(OutTag<OUT_F32>{}); break;
      case OUT_BF16: finish(OutTag<OUT_BF16>{}); break;
      case OUT_E4M3: finish(OutTag<OUT_E4M3>{}); break;
      default: finish(OutTag<OUT_NONE>{}); break;
    }
    if (RING) ring.next();
  }
  if (RING && bad && tid == 0) ring.drain((row - blockIdx.x) / step, (issued - blockIdx.x) / step, status);
  if (want_amax) {
    if (a.beside_zero) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (G == 1) {
      amax = warp_max(amax);
      if (tid == 0) atomic_max_nonneg(a.cast.amax_out, amax);
    } else {
      block_amax_commit(amax, a.cast.amax_out);
    }
  }
}

inline int round_warp(int64_t n) { return int((n + 31) / 32 * 32); }

__global__ void zero_scalar_kernel(float* p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  *p = 0.0f;
}

template <class K>
te_status launch_beside(K kernel, unsigned grid, int threads, size_t smem, const ResidualNormArgs& a, int slots,
                        cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.beside_zero ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, device_status_ptr(), slots) == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

template <typename TY, typename TR, bool LN, bool POST, int NV, int G>
te_status fwd_launch(const ResidualNormArgs& a, cudaStream_t s) {
  auto kernel = residual_norm_fwd_kernel<TY, TR, LN, POST, NV, G>;
  if constexpr (G == 0) {
    return launch_beside(kernel, unsigned(a.M), round_warp(a.H / 8), 0, a, 0, s);
  } else {
    static PerDevice<bool> attr_done;
    if (!allow_smem(kernel, attr_done)) return TE_ERR_CUDA;
    const size_t slot = size_t(a.H) * (sizeof(TY) + sizeof(TR));
    // three slots where L1 still holds the parameter vectors beside them (RMSNorm on both sides, 16384 x 4096:
    // 90 us for 97 with two; LayerNorm with a gate: 95 for 90)
    const size_t params = size_t(a.H) * sizeof(TY) * ((LN ? 2 : 1) * (POST ? 2 : 1) + (a.gate ? 1 : 0));
    const RingShape sh = ring_shape(fwd_ctas(G), slot, G > 1 && params <= 20 * 1024 ? 3 : 2);
    if (sh.ctas == 0) return TE_ERR_UNSUPPORTED;
    const int64_t n = int64_t(num_sms()) * sh.ctas;
    return launch_beside(kernel, unsigned(a.M < n ? a.M : n), G * 32, kHeader + size_t(sh.slots) * slot, a, sh.slots, s);
  }
}

template <typename TY, typename TR, bool LN, bool POST>
te_status fwd_shape(const ResidualNormArgs& a, cudaStream_t s) {
  const int64_t units = a.H / 8;
  // as long as every row has its CTA at once, latency counts: as many warps to a row as it has units
  if (units > 32 && a.M <= num_sms() * (units <= 512 ? 2 : 1)) return fwd_launch<TY, TR, LN, POST, 1, 0>(a, s);
  if (units <= 32) return fwd_launch<TY, TR, LN, POST, 1, 1>(a, s);
  if (units <= 64) return fwd_launch<TY, TR, LN, POST, 2, 1>(a, s);
  if (units <= 128) return fwd_launch<TY, TR, LN, POST, 4, 1>(a, s);
  if (units <= 256) return fwd_launch<TY, TR, LN, POST, 4, 2>(a, s);
  if (units <= 512) return fwd_launch<TY, TR, LN, POST, 4, 4>(a, s);
  return fwd_launch<TY, TR, LN, POST, 4, 8>(a, s);
}

template <typename TY, typename TR>
te_status fwd_types(const ResidualNormArgs& a, cudaStream_t s) {
  const bool post = a.post_gamma != nullptr;
  if (a.norm_type == TE_LAYERNORM)
    return post ? fwd_shape<TY, TR, true, true>(a, s) : fwd_shape<TY, TR, true, false>(a, s);
  return post ? fwd_shape<TY, TR, false, true>(a, s) : fwd_shape<TY, TR, false, false>(a, s);
}

}  // namespace

te_status launch_zero_scalar(float* p, cudaStream_t s) {
  zero_scalar_kernel<<<1, 1, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? TE_OK : TE_ERR_CUDA;
}

te_status launch_residual_norm_fwd(const ResidualNormArgs& a, cudaStream_t s) {
  if (a.M == 0) return TE_OK;
  ProfileScope prof(TE_KERNEL_NORM_FWD, s);
  if (a.y_dtype == TE_F32) return fwd_types<float, float>(a, s);
  return a.residual_dtype == TE_F32 ? fwd_types<__nv_bfloat16, float>(a, s)
                                    : fwd_types<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace te
