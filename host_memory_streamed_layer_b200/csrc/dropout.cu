// Dropout with a mask that is drawn again wherever it is needed, and the way
// back through a biased layer's dropout and activation (sm_100a):
//   y  = res + drop(x)
//   dz = drop(dc) act'(z),  db_j = sum over rows of dz_j (before dz is rounded)
// drop() zeroes an element or scales it by 1 / (1 - p). Both kernels are bound
// by device memory: each element is read and written once, eight at a time,
// and no mask is stored or read.
#include "act_dropout.cuh"

namespace mt {

namespace {

// Blocks of 256 threads: TX threads along a row (W columns each, 16 bytes of
// the wider type) by 256 / TX rows; grid.x covers the columns, grid.y the runs
// of rows. TX is the widest of 256, 128, 64, 32 that leaves the fewest threads
// without columns.
int pick_tx(int cols, int w) {
  const int pieces = (cols + w - 1) / w;
  int best = 32, waste = 1 << 30;
  for (int tx = 256; tx >= 32; tx >>= 1) {
    const int left = (pieces + tx - 1) / tx * tx - pieces;
    if (left < waste) waste = left, best = tx;
  }
  return best;
}

// Rows that a thread has in flight, W columns of each.
template <int W>
constexpr int ROWS = 8 / W;

template <int W>
__device__ __forceinline__ void drop_piece(float (&v)[W], int col, uint32_t row, const DropDesc& drop,
                                           const DropKey& key) {
#pragma unroll
  for (int h = 0; h < W / 4; ++h) drop4(v + 4 * h, (col >> 2) + h, row, drop, key);
}

// ROWS rows, ry apart, of one thread's columns. WHOLE: all of them are there and
// whole pieces, so that their loads go out together.
template <typename X, typename Y, int W, bool WHOLE>
__device__ __forceinline__ void dropout_rows(const X* x, int64_t ldx, const DropDesc& drop, const DropKey& key,
                                             const Y* res, int64_t ldr, Y* y, int64_t ldy, int64_t base, int ry, int T,
                                             int c, int n) {
  float v[ROWS<W>][W], r[ROWS<W>][W];
#pragma unroll
  for (int i = 0; i < ROWS<W>; ++i) {
    const int64_t t = base + i * ry;
    if (WHOLE || t < T) load_n<W>(x + t * ldx + c, WHOLE ? W : n, v[i]);
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < ROWS<W>; ++i) {
      const int64_t t = base + i * ry;
      if (WHOLE || t < T) load_n<W>(res + t * ldr + c, WHOLE ? W : n, r[i]);
    }
  }
  if (drop.on) {
#pragma unroll
    for (int i = 0; i < ROWS<W>; ++i) drop_piece<W>(v[i], c, drop.row0 + (uint32_t)(base + i * ry), drop, key);
  }
#pragma unroll
  for (int i = 0; i < ROWS<W>; ++i) {
    const int64_t t = base + i * ry;
    if (res) {
#pragma unroll
      for (int e = 0; e < W; ++e) v[i][e] += r[i][e];
    }
    if (WHOLE || t < T) store_n<W>(y + t * ldy + c, WHOLE ? W : n, v[i]);
  }
}

template <typename X, typename Y, int W>
__global__ void __launch_bounds__(256, 4) k_dropout(const X* x, int64_t ldx, const DropDesc drop, const Y* res, int64_t ldr,
                                                 Y* y, int64_t ldy, int T, int d, int tx_log2) {
  const int tx = threadIdx.x & ((1 << tx_log2) - 1), ry = 256 >> tx_log2;
  const int c = (((int)blockIdx.x << tx_log2) + tx) * W;
  if (c >= d) return;
  const int n = d - c;
  const DropKey key = drop_key(drop);
  const int64_t step = (int64_t)gridDim.y * ry * ROWS<W>;
  for (int64_t base = (int64_t)blockIdx.y * ry * ROWS<W> + (threadIdx.x >> tx_log2); base < T; base += step) {
    if (n >= W && base + (ROWS<W> - 1) * ry < T)
      dropout_rows<X, Y, W, true>(x, ldx, drop, key, res, ldr, y, ldy, base, ry, T, c, n);
    else
      dropout_rows<X, Y, W, false>(x, ldx, drop, key, res, ldr, y, ldy, base, ry, T, c, n);
  }
}

template <typename X, int ACT, int W, bool WHOLE>
__device__ __forceinline__ void act_bwd_rows(const X* dc, int64_t lddc, const bf16* z, int64_t ldz, const DropDesc& drop,
                                             const DropKey& key, bf16* dz, int64_t lddz, int64_t base, int ry,
                                             int64_t end, int c, int n, float (&acc)[W]) {
  float v[ROWS<W>][W], zv[ROWS<W>][W];
#pragma unroll
  for (int i = 0; i < ROWS<W>; ++i) {
    const int64_t t = base + i * ry;
    if (WHOLE || t < end) {
      load_n<W>(dc + t * lddc + c, WHOLE ? W : n, v[i]);
      if (ACT != MT_ACT_NONE) load_n<W>(z + t * ldz + c, WHOLE ? W : n, zv[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS<W>; ++i) {
    const int64_t t = base + i * ry;
    if (!WHOLE && t >= end) break;
    if (ACT != MT_ACT_NONE) {
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        const float2 slope = act_slope<ACT>(make_float2(zv[i][e], zv[i][e + 1]));
        v[i][e] *= slope.x, v[i][e + 1] *= slope.y;
      }
    }
    // last, so that a dropped element is 0 whatever dc and z hold there
    if (drop.on) drop_piece<W>(v[i], c, drop.row0 + (uint32_t)t, drop, key);
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] += v[i][e];
    store_n<W>(dz + t * lddz + c, WHOLE ? W : n, v[i]);
  }
}

template <typename X, int ACT, int W>
__global__ void __launch_bounds__(256, 4) k_act_bwd(const X* dc, int64_t lddc, const bf16* z, int64_t ldz,
                                                 const DropDesc drop, bf16* dz, int64_t lddz, float* __restrict__ part,
                                                 int M, int N, int rows_per_block, int tx_log2) {
  __shared__ float sh[256 * W];
  // The column sums' kernel starts once every block of this one has, so it takes
  // no room from them; up to 592 column strips they are all resident at once.
  let_next_start();
  const int TX = 1 << tx_log2, tx = threadIdx.x & (TX - 1), ty = threadIdx.x >> tx_log2, ry = 256 >> tx_log2;
  const int c = (((int)blockIdx.x << tx_log2) + tx) * W;
  const int n = N - c;
  const DropKey key = drop_key(drop);
  float acc[W];
#pragma unroll
  for (int e = 0; e < W; ++e) acc[e] = 0.f;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_block, r1 = min((int64_t)M, r0 + rows_per_block);
  if (n > 0) {
    for (int64_t base = r0 + ty; base < r1; base += ry * ROWS<W>) {
      if (n >= W && base + (ROWS<W> - 1) * ry < r1)
        act_bwd_rows<X, ACT, W, true>(dc, lddc, z, ldz, drop, key, dz, lddz, base, ry, r1, c, n, acc);
      else
        act_bwd_rows<X, ACT, W, false>(dc, lddc, z, ldz, drop, key, dz, lddz, base, ry, r1, c, n, acc);
    }
  }
  if (!part) return;
#pragma unroll
  for (int e = 0; e < W; ++e) sh[e * 256 + threadIdx.x] = acc[e];
  __syncthreads();
  // the block's rows in the order of ty; thread = (element e, column piece tx)
  for (int i = threadIdx.x; i < W * TX; i += 256) {
    const int e = i >> tx_log2, x = i & (TX - 1);
    float s = 0.f;
    for (int r = 0; r < ry; ++r) s += sh[e * 256 + (r << tx_log2) + x];
    const int col = (((int)blockIdx.x << tx_log2) + x) * W + e;
    if (col < N) part[(int64_t)blockIdx.y * N + col] = s;
  }
}

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

struct Grid {
  int tx_log2, gx, gy, rows_per_block;
};

// At most `blocks` blocks, and at least ROWS rows to a thread.
Grid grid_for(int rows, int cols, int w, int blocks) {
  Grid g;
  const int tx = pick_tx(cols, w), ry = 256 / tx, deep = 8 / w;
  g.tx_log2 = log2_of(tx);
  g.gx = ((cols + w - 1) / w + tx - 1) / tx;
  const int most = (rows + ry * deep - 1) / (ry * deep);
  const int want = blocks / g.gx > 1 ? blocks / g.gx : 1;
  g.gy = most < want ? most : want;
  if (g.gy > 65535) g.gy = 65535;
  if (g.gy < 1) g.gy = 1;
  g.rows_per_block = (rows + g.gy - 1) / g.gy;
  return g;
}

// Dropout: many short blocks, which leave no ragged last wave (8 to an SM took
// 84 us on 8192 x 5120 with a residual, 32 take 74).
constexpr int kDropoutBlocks = 148 * 32;
// The backward's blocks each leave a row of partial column sums, so there are
// only as many as run at once (one to each strip of columns at least).
constexpr int kActBwdBlocks = 148 * 4;

template <typename X, typename Y>
int dropout_launch(const void* x, int64_t ldx, const DropDesc& drop, const void* res, int64_t ldr, void* y, int64_t ldy,
                   int T, int d, cudaStream_t st) {
  constexpr int W = sizeof(X) == 4 || sizeof(Y) == 4 ? 4 : 8;
  const Grid g = grid_for(T, d, W, kDropoutBlocks);
  k_dropout<X, Y, W><<<dim3(g.gx, g.gy), 256, 0, st>>>((const X*)x, ldx, drop, (const Y*)res, ldr, (Y*)y, ldy, T, d,
                                                    g.tx_log2);
  return launch_status();
}

template <typename X>
int act_bwd_launch(const void* dc, int64_t lddc, const void* z, int64_t ldz, int act, const DropDesc& drop, void* dz,
                   int64_t lddz, float* part, float* db, int M, int N, cudaStream_t st) {
  constexpr int W = sizeof(X) == 4 ? 4 : 8;
  const Grid g = grid_for(M, N, W, kActBwdBlocks);
  float* p = db ? part : nullptr;
  MT_WITH_ACT(act, (k_act_bwd<X, ACT, W><<<dim3(g.gx, g.gy), 256, 0, st>>>((const X*)dc, lddc, (const bf16*)z, ldz, drop,
                                                                       (bf16*)dz, lddz, p, M, N, g.rows_per_block,
                                                                       g.tx_log2)));
  if (const int rc = launch_status()) return rc;
  return db ? launch_column_sums(part, g.gy, N, N, db, N, nullptr, st) : MT_OK;
}

}  // namespace

int launch_dropout(const void* x, int x_type, int64_t ldx, const DropDesc& drop, const void* res, int64_t ldr, void* y,
                   int y_type, int64_t ldy, int T, int d, cudaStream_t st) {
  if (T <= 0) return MT_OK;
  if (x_type == MT_F32 && y_type == MT_F32)
    return dropout_launch<float, float>(x, ldx, drop, res, ldr, y, ldy, T, d, st);
  if (x_type == MT_F32) return dropout_launch<float, bf16>(x, ldx, drop, res, ldr, y, ldy, T, d, st);
  if (y_type == MT_F32) return dropout_launch<bf16, float>(x, ldx, drop, res, ldr, y, ldy, T, d, st);
  return dropout_launch<bf16, bf16>(x, ldx, drop, res, ldr, y, ldy, T, d, st);
}

size_t act_bwd_partial_floats(int M, int N) {
  // dc's type is not known here
  const int a = grid_for(M, N, 4, kActBwdBlocks).gy, b = grid_for(M, N, 8, kActBwdBlocks).gy;
  return (size_t)(a > b ? a : b) * N;
}

int launch_act_bwd(const void* dc, int dc_type, int64_t lddc, const void* z, int64_t ldz, int act, const DropDesc& drop,
                   void* dz, int64_t lddz, float* part, float* db, int M, int N, cudaStream_t st) {
  if (N <= 0) return MT_OK;
  if (M <= 0) return !db || cudaMemsetAsync(db, 0, sizeof(float) * N, st) == cudaSuccess ? MT_OK : MT_ERR_CUDA;
  if (dc_type == MT_F32) return act_bwd_launch<float>(dc, lddc, z, ldz, act, drop, dz, lddz, part, db, M, N, st);
  return act_bwd_launch<bf16>(dc, lddc, z, ldz, act, drop, dz, lddz, part, db, M, N, st);
}

}  // namespace mt
