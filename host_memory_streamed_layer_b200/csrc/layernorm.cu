// Layer norm of a row, forward and backward (sm_100a):
//   y_j  = (x_j - m) r g_j + b_j,  m = mean x,  r = (mean (x - m)^2 + eps)^-1/2
// and, with w_j = dy_j g_j and xh_j = (x_j - m) r,
//   dx_j = dres_j + r (w_j - mean w - xh_j mean(w xh))
//   dg_j = sum over rows of dy_j xh_j,  db_j = sum over rows of dy_j.
// Both passes are bound by device memory: each reads its inputs once, and the
// row's two statistics are taken in fp32. The forward's first mean is off by the
// rounding of a sum of d values, a few 2^-24 of itself, which is much beside the
// spread of a row whose mean is large. So the centred values t = x - m are summed
// along with their squares: their mean s (nearly 0) is what m is off by, and
//   mean = m + s,  variance = mean t^2 - s^2,  xh = (t - s) r,
// where t itself is exact or nearly so. Measured on one B200: 16384 x 2048 fp32 to
// bf16 forward 37 us (5.4 TB/s), backward with the residual's gradient and a bf16
// copy 104 us (5.8 TB/s; a copy kernel reaches 6.5).
#include "act_dropout.cuh"

namespace mt {

namespace {

// Sum of (a, b) over the TX threads of a row piece; TX a multiple of 32. The
// block holds RY = blockDim.x / TX such rows; `red` has 2 * blockDim.x / 32
// floats. Every thread of the block calls it.
template <int TX>
__device__ __forceinline__ float2 row_sum2(float a, float b, float* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (TX == 32) return make_float2(a, b);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    red[2 * warp] = a;
    red[2 * warp + 1] = b;
  }
  __syncthreads();
  constexpr int W = TX / 32;
  const int w0 = warp / W * W;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    s.x += red[2 * (w0 + i)];
    s.y += red[2 * (w0 + i) + 1];
  }
  return s;
}

// The same for one number; `red` has blockDim.x / 32 floats.
template <int TX>
__device__ __forceinline__ float row_sum(float a, float* red) {
  a = warp_sum(a);
  if (TX == 32) return a;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = a;
  __syncthreads();
  constexpr int W = TX / 32;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) s += red[warp / W * W + i];
  return s;
}

// A lane reads W neighbouring columns at a time, 16 bytes of the wider of the
// two types: with eight columns of an fp32 row to a lane, each access would
// take only half of every sector that it touches.
template <typename X, typename Y>
constexpr int piece() {
  return sizeof(X) == 4 || sizeof(Y) == 4 ? 4 : 8;
}

// n columns from p on. EXACT: rows are whole pieces, so a piece is there or not
// and its load is one predicated instruction; with the element-wise tail beside
// it, each load would be a branch that the next one waits behind.
template <int W, bool EXACT, typename T>
__device__ __forceinline__ void load_piece(const T* p, int n, float (&v)[W]) {
  if (EXACT) {
    if (n > 0) {
      load_n<W>(p, W, v);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = 0.f;
    }
  } else {
    load_n<W>(p, n, v);
  }
}

// Forward: TX threads to a row, G pieces of W columns to a thread: 32 columns
// to a thread up to 4096, so that each has 64 bytes or more in flight (with 16
// columns a bf16 row of 2048 took 32.8 us for 16384 rows instead of 29.6). The
// arithmetic of two columns goes into one instruction: singly, the sum of t cost
// 2 to 9 % (bf16 16384 x 2048 32.8 us instead of 28.7; 30.8 without that sum). Eight
// columns to a thread leave room for eight blocks on an SM, 24 for five.
template <typename X, typename Y, int TX, int G, bool EXACT, int W = piece<X, Y>()>
__global__ void __launch_bounds__(256, G * W <= 8 ? 8 : EXACT && G * W <= 24 ? 5 : 4)
    k_layernorm_fwd(const X* __restrict__ x, int64_t ldx, const bf16* __restrict__ g, const bf16* __restrict__ b,
                    Y* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd, int T, int d,
                    float eps) {
  __shared__ float red[2][16];
  const int64_t row = (int64_t)blockIdx.x * (256 / TX) + threadIdx.x / TX;
  const int tx = threadIdx.x % TX;
  const bool ok = row < T;
  if (TX == 32 && !ok) return;  // a wider row's threads all stay for the barriers
  const X* xr = x + row * ldx;
  const float inv_d = 1.f / (float)d;
  float v[G][W];
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const int c = (tx + k * TX) * W;
    load_piece<W, EXACT>(xr + c, ok ? d - c : 0, v[k]);
  }
  // Sums of the even and of the odd columns.
  float2 s = make_float2(0.f, 0.f), u = s, q = s;
#pragma unroll
  for (int k = 0; k < G; ++k)
#pragma unroll
    for (int e = 0; e < W; e += 2) s = add2(s, make_float2(v[k][e], v[k][e + 1]));
  const float m = row_sum<TX>(s.x + s.y, red[0]) / (float)d;
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const int n = d - (tx + k * TX) * W;
    const float off = n > 0 ? -m : 0.f;  // behind the row: t = 0
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      const float2 t = add2(make_float2(v[k][e], v[k][e + 1]),
                            EXACT ? make_float2(off, off) : make_float2(e < n ? -m : 0.f, e + 1 < n ? -m : 0.f));
      u = add2(u, t);
      q = fma2(t, t, q);
      v[k][e] = t.x, v[k][e + 1] = t.y;
    }
  }
  const float2 tu = row_sum2<TX>(u.x + u.y, q.x + q.y, red[1]);
  const float shift = tu.x * inv_d, var = tu.y * inv_d - fminf(shift * shift, 3e38f);  // inf - inf: none
  const float r = rsqrtf((var < 0.f ? 0.f : var) + eps);  // below 0 by rounding alone; NaN stays
  const float minus = -shift * r;
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const int c = (tx + k * TX) * W;
    if (!ok || c >= d) continue;
    float gv[W], bv[W];
    load_n<W>(g + c, EXACT ? W : d - c, gv);
    if (b) {
      load_n<W>(b + c, EXACT ? W : d - c, bv);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) bv[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      const float2 xh = fma2(make_float2(v[k][e], v[k][e + 1]), make_float2(r, r), make_float2(minus, minus));
      const float2 o = fma2(xh, make_float2(gv[e], gv[e + 1]), make_float2(bv[e], bv[e + 1]));
      v[k][e] = o.x, v[k][e + 1] = o.y;
    }
    store_n<W>(y + row * ldy + c, EXACT ? W : d - c, v[k]);
  }
  if (ok && tx == 0) {
    if (mean) mean[row] = shift == shift ? m + shift : m;  // an infinite mean stays one
    if (rstd) rstd[row] = r;
  }
}

// Backward: a block takes a run of rows, RY at a time with TX threads to each;
// a thread keeps its columns' sums of dg and db over all of them. The block's
// sums go to its own row [dg | db] of `part`.
//
// Rows are copied into shared memory STAGES row groups ahead. A lane copies the
// very pieces that it reads back, so a copy needs no barrier, and the registers
// hold the sums instead of loads in flight: with the loads in registers,
// 8192 x 5120 took 155 us (one block to an SM), 16384 x 2048 took 110 us.
template <typename X, typename Y, int TX, int G>
struct LnBwd {
  static constexpr int W = piece<X, Y>();
  static constexpr int THREADS = TX > 256 ? TX : 256;
  static constexpr int RY = THREADS / TX;
  static constexpr int PX = W * sizeof(X), PY = W * sizeof(Y);  // bytes of a piece
  static constexpr int ROWS_BYTES = THREADS * G * (2 * PX + PY);  // x, dres and dy of a row group
  static constexpr int STAGES = ROWS_BYTES <= 75776 ? 3 : 2;
  static constexpr int SMEM = STAGES * ROWS_BYTES;
  static constexpr int PER_SM = SMEM <= 74 * 1024 && THREADS == 256 ? 3 : SMEM <= 112 * 1024 ? 2 : 1;
};

template <typename T, int W>
__device__ __forceinline__ void copy_piece(uint32_t dst, const T* src) {
  if (W * sizeof(T) == 16)
    copy16(dst, src);
  else
    copy8(dst, src);
}

template <typename X, typename Y, int TX, int G, bool EXACT>
__global__ void __launch_bounds__(LnBwd<X, Y, TX, G>::THREADS, LnBwd<X, Y, TX, G>::PER_SM)
    k_layernorm_bwd(const X* x, int64_t ldx, const bf16* __restrict__ g, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const Y* dy, int64_t lddy, const X* dres, int64_t lddres, X* dx,
                    bf16* dx_bf16, int64_t lddx, float* __restrict__ part, int T, int d, int rows_per_block) {
  using L = LnBwd<X, Y, TX, G>;
  constexpr int W = L::W, RY = L::RY, S = L::STAGES;
  extern __shared__ __align__(16) uint8_t ring[];
  let_next_start();  // the column sums' kernel; every block of this one is resident from the start
  __shared__ float red[2][L::THREADS / 16];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  float ag[G][W], ab[G][W], gv[G][W];
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const int c = (tx + k * TX) * W;
    load_piece<W, EXACT>(g + c, d - c, gv[k]);
#pragma unroll
    for (int e = 0; e < W; ++e) ag[k][e] = ab[k][e] = 0.f;
  }
  const int64_t r0 = (int64_t)blockIdx.x * rows_per_block;
  const int64_t r1 = min((int64_t)T, r0 + rows_per_block);
  const int groups = r1 > r0 ? (int)((r1 - r0 + RY - 1) / RY) : 0;
  // This lane's slots of a stage: G pieces of x, of dres, of dy.
  const uint32_t mine = smem_u32(ring) + threadIdx.x * L::PX;
  const uint32_t mine_y = smem_u32(ring) + L::THREADS * G * 2 * L::PX + threadIdx.x * L::PY;
  auto fetch = [&](int i) {  // row group i, one group of copies (empty behind the last)
    const int64_t row = r0 + (int64_t)i * RY + ty;
    if (EXACT && i < groups && row < r1) {
      const uint32_t at = i % S * L::ROWS_BYTES;
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int c = (tx + k * TX) * W;
        if (c >= d) break;
        copy_piece<X, W>(mine + at + k * L::THREADS * L::PX, x + row * ldx + c);
        copy_piece<Y, W>(mine_y + at + k * L::THREADS * L::PY, dy + row * lddy + c);
        if (dres) copy_piece<X, W>(mine + at + (G + k) * L::THREADS * L::PX, dres + row * lddres + c);
      }
    }
    copy_commit();
  };
  if (EXACT) {
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);
  }
  float next_m = 0.f, next_r = 0.f;
  if (r0 + ty < r1) next_m = mean[r0 + ty], next_r = rstd[r0 + ty];
  for (int i = 0; i < groups; ++i) {
    const int64_t row = r0 + (int64_t)i * RY + ty;
    const bool ok = row < r1;
    const float m = next_m, r = next_r;
    if (row + RY < r1) next_m = mean[row + RY], next_r = rstd[row + RY];
    float xv[G][W], dv[G][W], rv[G][W];
    if (EXACT) {
      fetch(i + S - 1);
      copy_wait<S - 1>();
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int c = (tx + k * TX) * W, n = ok ? d - c : 0;
      if (EXACT) {
        const uint8_t* stage = ring + i % S * L::ROWS_BYTES;
        const uint8_t* at = stage + k * L::THREADS * L::PX + threadIdx.x * L::PX;
        const uint8_t* at_y = stage + L::THREADS * (G * 2 * L::PX + k * L::PY) + threadIdx.x * L::PY;
        load_piece<W, true>(reinterpret_cast<const X*>(at), n, xv[k]);
        load_piece<W, true>(reinterpret_cast<const Y*>(at_y), n, dv[k]);
        if (dres) load_piece<W, true>(reinterpret_cast<const X*>(at + G * L::THREADS * L::PX), n, rv[k]);
      } else {
        load_n<W>(x + row * ldx + c, n, xv[k]);
        load_n<W>(dy + row * lddy + c, n, dv[k]);
        if (dres) load_n<W>(dres + row * lddres + c, n, rv[k]);
      }
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int n = d - (tx + k * TX) * W;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float xh = ok && (EXACT ? n > 0 : e < n) ? (xv[k][e] - m) * r : 0.f;
        const float w = dv[k][e] * gv[k][e];
        xv[k][e] = xh;
        s1 += w;
        s2 += w * xh;
        ag[k][e] += dv[k][e] * xh;
        ab[k][e] += dv[k][e];
      }
    }
    const float2 s = row_sum2<TX>(s1, s2, red[i & 1]);  // the halves alternate: one barrier a row group
    const float m1 = s.x / (float)d, m2 = s.y / (float)d;
    if (ok) {
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int c = (tx + k * TX) * W;
        if (c >= d) continue;
        float o[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          o[e] = r * (dv[k][e] * gv[k][e] - m1 - xv[k][e] * m2);
          if (dres) o[e] += rv[k][e];
        }
        store_n<W>(dx + row * lddx + c, EXACT ? W : d - c, o);
        if (dx_bf16) store_n<W>(dx_bf16 + row * lddx + c, EXACT ? W : d - c, o);
      }
    }
  }
  copy_wait<0>();
  // The RY rows' sums meet in shared memory, in the order of ty: dg, then db.
  float* col = reinterpret_cast<float*>(ring);  // [RY - 1][G W][TX], at most as large as a stage
  float* out = part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float(&acc)[G][W] = which ? ab : ag;
    if (RY > 1) {
      __syncthreads();
      if (ty > 0) {
#pragma unroll
        for (int k = 0; k < G; ++k)
#pragma unroll
          for (int e = 0; e < W; ++e) col[((ty - 1) * G * W + k * W + e) * TX + tx] = acc[k][e];
      }
      __syncthreads();
    }
    if (ty == 0) {
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int c = (tx + k * TX) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          float s = acc[k][e];
#pragma unroll
          for (int i = 0; i < RY - 1; ++i) s += col[(i * G * W + k * W + e) * TX + tx];
          if (c + e < d) out[which * d + c + e] = s;
        }
      }
    }
  }
}

// out[j] = sum over r of part[r, j], 32 columns to a block; thread row y takes
// the partials y, y + 32, ... and the 32 sums meet in a fixed tree.
__global__ void __launch_bounds__(1024) k_column_sums(const float* __restrict__ part, int rows, int64_t pitch, int n,
                                                      float* __restrict__ out, int n1, float* __restrict__ out2) {
  __shared__ float sh[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + x;
  float s = 0.f;
  wait_for_previous();
  if (j < n) {
#pragma unroll 4
    for (int r = y; r < rows; r += 32) s += part[(int64_t)r * pitch + j];
  }
  sh[y][x] = s;
  __syncthreads();
  const float t = warp_sum(sh[x][y]);  // warp y now holds column y's 32 sums
  const int o = blockIdx.x * 32 + y;
  if (x == 0 && o < n) {
    if (o < n1)
      out[o] = t;
    else if (out2)
      out2[o - n1] = t;
  }
}

// The backward's blocks: as many as run at once on 148 SMs, fewer where a block
// would have less than two row groups. Three to an SM bounds the scratch.
constexpr int kLnMaxBlocks = 3 * 148;

int ln_bwd_blocks(int T, int per_sm, int ry) {
  const int64_t most = ((int64_t)T + 2 * ry - 1) / (2 * ry);
  return (int)(most < per_sm * 148 ? most : per_sm * 148);
}

template <typename X, typename Y, int TX, int G>
int ln_fwd_launch(const void* x, int64_t ldx, const void* g, const void* b, void* y, int64_t ldy, float* mean,
                  float* rstd, int T, int d, float eps, cudaStream_t st) {
  const int rpb = 256 / TX;
  auto k = d % piece<X, Y>() ? k_layernorm_fwd<X, Y, TX, G, false> : k_layernorm_fwd<X, Y, TX, G, true>;
  k<<<(T + rpb - 1) / rpb, 256, 0, st>>>((const X*)x, ldx, (const bf16*)g, (const bf16*)b, (Y*)y, ldy, mean, rstd, T, d,
                                         eps);
  return launch_status();
}

template <typename X, typename Y>
int ln_fwd(const void* x, int64_t ldx, const void* g, const void* b, void* y, int64_t ldy, float* mean, float* rstd,
           int T, int d, float eps, cudaStream_t st) {
  constexpr int P = 8 / piece<X, Y>();  // pieces of a lane for each eight columns
#define MT_LN_FWD(TX, G) return ln_fwd_launch<X, Y, TX, G * P>(x, ldx, g, b, y, ldy, mean, rstd, T, d, eps, st)
  if (d <= 256) MT_LN_FWD(32, 1);
  if (d <= 512) MT_LN_FWD(32, 2);
  if (d <= 1024) MT_LN_FWD(32, 4);
  if (d <= 2048) MT_LN_FWD(64, 4);
  if (d <= 4096) MT_LN_FWD(128, 4);
  if (d <= 6144) MT_LN_FWD(256, 3);
  MT_LN_FWD(256, 4);
#undef MT_LN_FWD
}

template <typename X, typename Y, int TX, int G>
int ln_bwd_launch(const LayerNormBwd& a, cudaStream_t st) {
  using L = LnBwd<X, Y, TX, G>;
  const int nb = ln_bwd_blocks(a.T, L::PER_SM, L::RY);
  const int rpb = (a.T + nb - 1) / nb;
  auto k = a.d % L::W ? k_layernorm_bwd<X, Y, TX, G, false> : k_layernorm_bwd<X, Y, TX, G, true>;
  // Above 48 KB a kernel has to be told, once on each device.
  static bool told[2][kMaxDevices] = {};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device >= kMaxDevices) return MT_ERR_CUDA;
  bool& is = told[a.d % L::W ? 1 : 0][device];
  if (!is && cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM) != cudaSuccess)
    return MT_ERR_CUDA;
  is = true;
  k<<<nb, L::THREADS, L::SMEM, st>>>((const X*)a.x, a.ldx, (const bf16*)a.g, a.mean, a.rstd, (const Y*)a.dy, a.lddy,
                                     (const X*)a.dres, a.lddres, (X*)a.dx, (bf16*)a.dx_bf16, a.lddx, a.part, a.T, a.d,
                                     rpb);
  if (const int rc = launch_status()) return rc;
  return launch_column_sums(a.part, nb, 2 * (int64_t)a.d, 2 * a.d, a.dg, a.d, a.db, st);
}

template <typename X, typename Y>
int ln_bwd(const LayerNormBwd& a, cudaStream_t st) {
  constexpr int P = 8 / piece<X, Y>();
  if (a.d <= 256) return ln_bwd_launch<X, Y, 32, P>(a, st);
  if (a.d <= 512) return ln_bwd_launch<X, Y, 64, P>(a, st);
  if (a.d <= 1024) return ln_bwd_launch<X, Y, 128, P>(a, st);
  if (a.d <= 2048) return ln_bwd_launch<X, Y, 256, P>(a, st);
  if (a.d <= 4096) return ln_bwd_launch<X, Y, 512, P>(a, st);
  if (P == 2 && a.d <= 6144) return ln_bwd_launch<X, Y, 512, P + P / 2>(a, st);
  return ln_bwd_launch<X, Y, 512, 2 * P>(a, st);
}

}  // namespace

int launch_column_sums(const float* part, int rows, int64_t pitch, int n, float* out, int n1, float* out2,
                       cudaStream_t st) {
  if (n <= 0) return MT_OK;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((n + 31) / 32, 1, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, k_column_sums, part, rows, pitch, n, out, n1, out2);
  return launch_status();
}

int launch_layernorm_fwd(const void* x, int x_type, int64_t ldx, const void* g, const void* b, void* y, int y_type,
                         int64_t ldy, float* mean, float* rstd, int T, int d, float eps, cudaStream_t st) {
  if (T <= 0) return MT_OK;
  if (x_type == MT_F32 && y_type == MT_F32)
    return ln_fwd<float, float>(x, ldx, g, b, y, ldy, mean, rstd, T, d, eps, st);
  if (x_type == MT_F32) return ln_fwd<float, bf16>(x, ldx, g, b, y, ldy, mean, rstd, T, d, eps, st);
  if (y_type == MT_F32) return ln_fwd<bf16, float>(x, ldx, g, b, y, ldy, mean, rstd, T, d, eps, st);
  return ln_fwd<bf16, bf16>(x, ldx, g, b, y, ldy, mean, rstd, T, d, eps, st);
}

size_t layernorm_bwd_partial_floats(int T, int d) { return (size_t)(T < kLnMaxBlocks ? T + 1 : kLnMaxBlocks) * 2 * d; }

int launch_layernorm_bwd(const LayerNormBwd& a, cudaStream_t st) {
  if (a.T <= 0) {  // sums over no rows
    if (cudaMemsetAsync(a.dg, 0, sizeof(float) * a.d, st) != cudaSuccess) return MT_ERR_CUDA;
    if (a.db && cudaMemsetAsync(a.db, 0, sizeof(float) * a.d, st) != cudaSuccess) return MT_ERR_CUDA;
    return MT_OK;
  }
  if (a.x_type == MT_F32 && a.dy_type == MT_F32) return ln_bwd<float, float>(a, st);
  if (a.x_type == MT_F32) return ln_bwd<float, bf16>(a, st);
  if (a.dy_type == MT_F32) return ln_bwd<bf16, float>(a, st);
  return ln_bwd<bf16, bf16>(a, st);
}

}  // namespace mt
