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

// Blocks of 256 threads: TX threads along a row (eight columns each) by
// 256 / TX rows; grid.x covers the columns, grid.y the runs of rows. TX is
// the widest of 256, 128, 64, 32 that leaves the fewest threads without columns.
int pick_tx(int cols) {
  const int pieces = (cols + 7) / 8;
  int best = 32, waste = 1 << 30;
  for (int tx = 256; tx >= 32; tx >>= 1) {
    const int w = (pieces + tx - 1) / tx * tx - pieces;
    if (w < waste) waste = w, best = tx;
  }
  return best;
}

constexpr int ROWS = 4;  // rows that a thread has in flight

template <typename X, typename Y>
__global__ void __launch_bounds__(256) k_dropout(const X* x, int64_t ldx, const DropDesc drop, const Y* res, int64_t ldr,
                                                 Y* y, int64_t ldy, int T, int d, int tx_log2) {
  const int tx = threadIdx.x & ((1 << tx_log2) - 1), ry = 256 >> tx_log2;
  const int c = (((int)blockIdx.x << tx_log2) + tx) * 8;
  if (c >= d) return;
  const int n = d - c;
  const DropKey key = drop_key(drop);
  const int64_t step = (int64_t)gridDim.y * ry * ROWS;
  for (int64_t base = (int64_t)blockIdx.y * ry * ROWS + (threadIdx.x >> tx_log2); base < T; base += step) {
    float v[ROWS][8], r[ROWS][8];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int64_t t = base + i * ry;
      if (t < T) {
        load8n(x + t * ldx + c, n, v[i]);
        if (res) load8n(res + t * ldr + c, n, r[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int64_t t = base + i * ry;
      if (t >= T) break;
      if (drop.on) {
        drop4(v[i], c >> 2, drop.row0 + (uint32_t)t, drop, key);
        drop4(v[i] + 4, (c >> 2) + 1, drop.row0 + (uint32_t)t, drop, key);
      }
      if (res) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] += r[i][e];
      }
      store8n(y + t * ldy + c, n, v[i]);
    }
  }
}

template <typename X, int ACT>
__global__ void __launch_bounds__(256) k_act_bwd(const X* __restrict__ dc, int64_t lddc, const bf16* __restrict__ z,
                                                 int64_t ldz, const DropDesc drop, bf16* __restrict__ dz, int64_t lddz,
                                                 float* __restrict__ part, int M, int N, int rows_per_block,
                                                 int tx_log2) {
  __shared__ float sh[256 * 8];
  const int TX = 1 << tx_log2, tx = threadIdx.x & (TX - 1), ty = threadIdx.x >> tx_log2, ry = 256 >> tx_log2;
  const int c = (((int)blockIdx.x << tx_log2) + tx) * 8;
  const int n = N - c;
  const DropKey key = drop_key(drop);
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_block, r1 = min((int64_t)M, r0 + rows_per_block);
  if (n > 0) {
    for (int64_t base = r0 + ty; base < r1; base += ry * ROWS) {
      float v[ROWS][8], zv[ROWS][8];
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int64_t t = base + i * ry;
        if (t < r1) {
          load8n(dc + t * lddc + c, n, v[i]);
          if (ACT != MT_ACT_NONE) load8n(z + t * ldz + c, n, zv[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int64_t t = base + i * ry;
        if (t >= r1) break;
        if (ACT != MT_ACT_NONE) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] *= act_slope<ACT>(zv[i][e]);
        }
        if (drop.on) {  // last, so that a dropped element is 0 whatever dc and z hold there
          drop4(v[i], c >> 2, drop.row0 + (uint32_t)t, drop, key);
          drop4(v[i] + 4, (c >> 2) + 1, drop.row0 + (uint32_t)t, drop, key);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += v[i][e];
        store8n(dz + t * lddz + c, n, v[i]);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sh[e * 256 + threadIdx.x] = acc[e];
  __syncthreads();
  // the block's rows in the order of ty; thread = (element e, column piece tx)
  for (int i = threadIdx.x; i < 8 * TX; i += 256) {
    const int e = i >> tx_log2, x = i & (TX - 1);
    float s = 0.f;
    for (int r = 0; r < ry; ++r) s += sh[e * 256 + (r << tx_log2) + x];
    const int col = (((int)blockIdx.x << tx_log2) + x) * 8 + e;
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

// About 8 blocks for each of 148 SMs, and at least ROWS rows to a thread.
Grid grid_for(int rows, int cols) {
  Grid g;
  const int tx = pick_tx(cols), ry = 256 / tx;
  g.tx_log2 = log2_of(tx);
  g.gx = ((cols + 7) / 8 + tx - 1) / tx;
  const int most = (rows + ry * ROWS - 1) / (ry * ROWS);
  const int want = (148 * 8 + g.gx - 1) / g.gx;
  g.gy = most < want ? most : want;
  if (g.gy > 1024) g.gy = 1024;
  if (g.gy < 1) g.gy = 1;
  g.rows_per_block = (rows + g.gy - 1) / g.gy;
  return g;
}

template <typename X, typename Y>
int dropout_launch(const void* x, int64_t ldx, const DropDesc& drop, const void* res, int64_t ldr, void* y, int64_t ldy,
                   int T, int d, cudaStream_t st) {
  const Grid g = grid_for(T, d);
  k_dropout<X, Y><<<dim3(g.gx, g.gy), 256, 0, st>>>((const X*)x, ldx, drop, (const Y*)res, ldr, (Y*)y, ldy, T, d,
                                                    g.tx_log2);
  return launch_status();
}

template <typename X>
int act_bwd_launch(const void* dc, int64_t lddc, const void* z, int64_t ldz, int act, const DropDesc& drop, void* dz,
                   int64_t lddz, float* part, float* db, int M, int N, cudaStream_t st) {
  const Grid g = grid_for(M, N);
  float* p = db ? part : nullptr;
  MT_WITH_ACT(act, (k_act_bwd<X, ACT><<<dim3(g.gx, g.gy), 256, 0, st>>>((const X*)dc, lddc, (const bf16*)z, ldz, drop,
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

size_t act_bwd_partial_floats(int M, int N) { return (size_t)grid_for(M, N).gy * N; }

int launch_act_bwd(const void* dc, int dc_type, int64_t lddc, const void* z, int64_t ldz, int act, const DropDesc& drop,
                   void* dz, int64_t lddz, float* part, float* db, int M, int N, cudaStream_t st) {
  if (N <= 0) return MT_OK;
  if (M <= 0) return !db || cudaMemsetAsync(db, 0, sizeof(float) * N, st) == cudaSuccess ? MT_OK : MT_ERR_CUDA;
  if (dc_type == MT_F32) return act_bwd_launch<float>(dc, lddc, z, ldz, act, drop, dz, lddz, part, db, M, N, st);
  return act_bwd_launch<bf16>(dc, lddc, z, ldz, act, drop, dz, lddz, part, db, M, N, st);
}

}  // namespace mt
